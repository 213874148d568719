"""GPU parity of the block operators against the fp64 oracle (oracle/block.py).

Tolerances.  u = 2^-24 is half an fp32 step relative to the value, 2^-8 half a bf16 one.
  * Picks: the operator's choice is that of fp64 scores, as the oracle's; they are equal unless two
    scores are within about 2^-50 of each other, which no input here has but by an exact tie.
  * A share of the picks is exp(ls - top) / sum: ls = log s is off by at most 4 u |ls| + 4 u (a
    difference of a minimum and log1p(exp)), top alike, exp by 2 u, the sum of at most 64 by 8 u,
    the quotient and the scale by 2 u: 8 max|ls| + 32 of u.  A softmax probability as in the balance
    loss's tests: (|l - m| + 80) u p.
  * The gradient of a pick is made of two such shares, a sum of at most 64 products and a few
    products: C = 16 max|ls| + 256 of u, relative to the sum of the absolute values of its terms.
  * A sum of c terms along a chain is off by at most (c + 2) u of the sum of absolute values.  A row
    of the norms: 8 to 32 elements a thread, 6 steps across a wave, at most 16 waves: 60 u; the root
    halves it, its reciprocal adds 2 u.
  * FP8 codes and exponents are exact.  A product is off by the matrix cores' sums, 2^-11 (|C| + rss
    of its products) (four times the largest seen by the FP8 layer's tests), and its rounding.
Each bound below is such a sum; none is fitted to a result.
"""
import numpy as np
import pytest

from gpu_common import device, say, to_np
from oracle import block as ob

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def put(a, dtype=None):
    import torch
    t = torch.tensor(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(device())


def tdtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def stored(a, name):
    """(tensor on the device, its exact values)."""
    t = put(np.asarray(a, np.float32), tdtype(name))
    return t, t.double().cpu().numpy()


def f64(t):
    return t.double().cpu().numpy()


def lm():
    import mixture_experts_layer_router_amd
    return mixture_experts_layer_router_amd


# ---- choice of experts ------------------------------------------------------------------------

SEL = [dict(T=1, E=1, K=1), dict(T=1, E=7, K=7), dict(T=5, E=12, K=2, score="sigmoid"),
       dict(T=65, E=768, K=12, renorm=True, pad=0.2), dict(T=64, E=768, K=12, score="sigmoid", groups=8, top_groups=4,
                                                         group_rank=2, renorm=True, scale=2.5),
       dict(T=33, E=96, K=6, groups=6, top_groups=2, group_rank=1, off=0.3),
       dict(T=40, E=96, K=6, score="sigmoid", groups=3, top_groups=1, group_rank=2, off=0.7, pad=0.3),
       dict(T=19, E=77, K=5, renorm=True, scale=0.5), dict(T=9, E=64, K=64, score="sigmoid", renorm=True),
       dict(T=9, E=64, K=8, groups=64, top_groups=8), dict(T=7, E=4096, K=16, groups=32, top_groups=5, group_rank=2,
                                                        renorm=True),
       dict(T=3, E=4095, K=64, score="sigmoid"), dict(T=21, E=130, K=12, groups=2, top_groups=1, group_rank=2, nobias=True),
       dict(T=300, E=260, K=8, groups=4, top_groups=2, group_rank=2, score="sigmoid", renorm=True),
       dict(T=17, E=63, K=9, groups=7, top_groups=3, off=0.5), dict(T=1030, E=16, K=4, renorm=True)]


def gating_of(kw):
    return {k: kw[k] for k in ("score", "groups", "top_groups", "group_rank", "renorm", "scale") if k in kw}


def select_inputs(kw, seed=3, spread=1.5):
    T, E = kw["T"], kw["E"]
    rng = np.random.default_rng(seed)
    lg = (spread * rng.standard_normal((T, E))).astype(np.float32)
    b = None if kw.get("nobias") else (0.05 * rng.uniform(-1, 1, E)).astype(np.float32)
    if "off" in kw:
        lg[rng.random((T, E)) < kw["off"]] = -np.inf
        b[rng.random(E) < kw["off"] / 3] = -np.inf
        lg[0] = -np.inf
    mask = (rng.random(T) >= kw["pad"]).astype(np.uint8) if "pad" in kw else None
    return lg, b, mask


def ls_bound(lg, idx, score):
    """Largest |log s| among the picks."""
    ls = np.abs(np.take_along_axis(ob.log_scores(lg, score), np.maximum(idx, 0), 1))
    return float(np.where((idx >= 0) & np.isfinite(ls), ls, 0).max())


def check_select(kw, lg, b, mask, got):
    g = gating_of(kw)
    idx, gate = ob.select(lg, b, kw["K"], mask=mask, **g)
    np.testing.assert_array_equal(to_np(got[0]), idx)
    score = g.get("score", "softmax")
    if g.get("renorm"):
        tol = (8 * ls_bound(lg, idx, score) + 32) * U
    else:
        top = np.where(np.isfinite(lg), lg, -np.inf).max(1, keepdims=True)
        d = np.where(np.isfinite(top), top, 0) - np.take_along_axis(lg, np.maximum(idx, 0), 1)
        tol = (np.abs(np.where(np.isfinite(d), d, 0)).max() + 80) * U
    np.testing.assert_allclose(to_np(got[1]), gate, rtol=tol, atol=2.0 ** -126)
    return idx, gate


@pytest.mark.parametrize("kw", SEL, ids=lambda k: "_".join(f"{a}{v}" for a, v in k.items()))
def test_select(kw):
    import torch
    say(f"select {kw}")
    lg, b, mask = select_inputs(kw)
    args = (put(lg), None if b is None else put(b), kw["K"], lm().Gating(**gating_of(kw)))
    tm = None if mask is None else put(mask)
    got = lm().select(*args, token_mask=tm)
    check_select(kw, lg, b, mask, got)
    again = lm().select(*args, token_mask=tm)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_select_ties(score, groups):
    """Equal scores, a whole row of them too: the lower expert and the lower group first."""
    say(f"select ties {score} {groups}")
    rng = np.random.default_rng(5)
    T, E, K = 70, 64, 10
    lg = rng.integers(-2, 3, (T, E)).astype(np.float32)
    lg[0] = 0.0
    lg[1] = -80.0
    lg[2, ::2] = -np.inf
    kw = dict(K=K, score=score, groups=groups, top_groups=max(groups // 2, 1), group_rank=2 if groups > 1 else 1)
    for b in (None, np.zeros(E, np.float32), np.full(E, -0.25, np.float32)):
        got = lm().select(put(lg), None if b is None else put(b), K, lm().Gating(**gating_of(kw)))
        check_select(kw, lg, b, None, got)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 8])
def test_select_next_to_a_border(score, groups):
    """Scores that fp32 cannot tell apart: logits one step apart, and biases that make up for a
    difference of scores but for its last digits.  fp64 decides."""
    say(f"select borders {score} {groups}")
    rng = np.random.default_rng(11)
    T, E, K = 200, 64, 6
    lg = rng.standard_normal((T, E)).astype(np.float32)
    b = (0.01 * rng.standard_normal(E)).astype(np.float32)
    for t in range(T):  # half of a token's experts are next to another's
        order = rng.permutation(E)
        for i, j in zip(order[:16], order[16:32]):
            lg[t, j] = np.nextafter(lg[t, i], np.float32(9), dtype=np.float32)
    b[:] = b[0]
    b[5] = np.float32(0.3)
    lg[3, 5] = -4.0
    kw = dict(K=K, score=score, groups=groups, top_groups=max(groups // 2, 1), group_rank=2 if groups > 1 else 1)
    got = lm().select(put(lg), put(b), K, lm().Gating(**gating_of(kw)))
    check_select(kw, lg, b, None, got)


LOWEST = np.finfo(np.float32).min


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,rank", [(1, 1), (4, 1), (4, 2), (8, 2)])
@pytest.mark.parametrize("E", [64, 96, 768])
def test_select_lowest_values(score, groups, rank, E):
    """Masks of fp32's lowest value, in logits and biases, rows of nothing else too: such an expert is on, after
    all that are larger and ahead of those that are off."""
    say(f"select lowest values {score} {groups} {rank} {E}")
    rng = np.random.default_rng(17)
    T, K, size = 24, 8, E // groups
    lg = rng.standard_normal((T, E)).astype(np.float32)
    lg[0] = LOWEST
    lg[1, 3:] = LOWEST
    lg[2, :E // 2] = LOWEST
    lg[3, rng.random(E) < 0.9] = LOWEST
    lg[4] = LOWEST
    lg[4, ::2] = -np.inf
    lg[5] = LOWEST / 2
    lg[6] = -1e30
    lg[7] = np.linspace(-95, -80, E)
    lg[8, :size] = -np.inf
    lg[9] = LOWEST
    lg[9, E - size:] = -np.inf
    kw = dict(K=K, score=score, groups=groups, top_groups=max(groups // 2, 1), group_rank=rank)
    plain = (0.05 * rng.uniform(-1, 1, E)).astype(np.float32)
    low, some, half, high = plain.copy(), plain.copy(), plain.copy(), plain.copy()
    low[:] = LOWEST
    some[size // 2:] = LOWEST
    half[:E // 2], half[E // 2:] = LOWEST / 2, LOWEST
    high[::3] = -LOWEST
    off = low.copy()
    off[:size] = -np.inf
    for b in (None, plain, low, some, half, high, off):
        for renorm in (False, True):
            kw["renorm"] = renorm
            got = lm().select(put(lg), None if b is None else put(b), K, lm().Gating(**gating_of(kw)))
            idx, gate = ob.select(lg, b, **kw)
            np.testing.assert_array_equal(to_np(got[0]), idx)
            # logits of a token are equal, or within 100 of 0, or so far below its largest that their scores
            # are less than 2^-126 of it
            np.testing.assert_allclose(to_np(got[1]), gate, rtol=(8 * 150 + 80) * U, atol=2.0 ** -126)


def test_select_far_logits():
    """Scores far below fp32's range still have shares, and large ones saturate without NaN."""
    say("select far logits")
    rng = np.random.default_rng(7)
    lg = (40 * rng.standard_normal((50, 96))).astype(np.float32)
    lg[0] -= 400
    lg[1] = np.linspace(-300, -200, 96)
    for score in ("softmax", "sigmoid"):
        kw = dict(K=8, score=score, renorm=True)
        # a bias that picks experts of hardly any score
        b = np.where(np.arange(96) % 5 == 0, 2.0, 0.0).astype(np.float32) + np.arange(96, dtype=np.float32) / 1024
        got = lm().select(put(lg), put(b), 8, lm().Gating(**gating_of(kw)))
        check_select(kw, lg, b, None, got)


BW = [dict(T=1, E=1, K=1), dict(T=6, E=12, K=3, score="sigmoid"), dict(T=65, E=768, K=12, renorm=True, aux=True),
      dict(T=64, E=768, K=12, score="sigmoid", renorm=True, scale=2.5, aux=True), dict(T=31, E=77, K=5, aux=True, scale=0.5),
      dict(T=10, E=77, K=5, renorm=True), dict(T=5, E=4096, K=64), dict(T=5, E=4095, K=64, score="sigmoid", renorm=True),
      dict(T=40, E=30, K=8, repeat=True), dict(T=40, E=30, K=8, repeat=True, renorm=True, aux=True),
      dict(T=40, E=30, K=8, repeat=True, score="sigmoid"), dict(T=515, E=96, K=6, renorm=True)]


@pytest.mark.parametrize("kw", BW, ids=lambda k: "_".join(f"{a}{v}" for a, v in k.items()))
def test_select_backward(kw):
    import torch
    say(f"select backward {kw}")
    T, E, K = kw["T"], kw["E"], kw["K"]
    rng = np.random.default_rng(2)
    lg = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    if kw.get("repeat"):
        idx = rng.integers(-1, E + 1, (T, K))  # repeated ones and ones outside the pool
        idx[0] = -1
        idx[1] = 4
    else:
        idx = np.argsort(rng.random((T, E)), 1)[:, :K]
    dg = rng.standard_normal((T, K)).astype(np.float32)
    aux = (0.1 * rng.standard_normal((T, E))).astype(np.float32) if kw.get("aux") else None
    g = gating_of(kw)
    ref, mag = ob.select_backward(lg, idx, dg, g.get("score", "softmax"), g.get("renorm", False), g.get("scale", 1.0), aux)
    args = (put(lg), put(idx.astype(np.int32)), put(dg), lm().Gating(**g), None if aux is None else put(aux))
    got = lm().select_backward(*args)
    inside = np.where((idx >= 0) & (idx < E), idx, -1)
    C = 16 * max(ls_bound(lg, inside, g.get("score", "softmax")), 12) + 256
    over = np.abs(f64(got) - ref) - C * U * mag
    assert over.max() <= 1e-37, over.max()
    assert torch.equal(got, lm().select_backward(*args))


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_select_backward_against_differences(score, renorm):
    """Central differences of the operator's own gates.  Their step of 2^-6 leaves an error of
    step^2 / 6 times the third derivative (at most 1 for these functions of scale 1), and the
    gates' rounding over twice the step."""
    import torch
    say(f"select differences {score} {renorm}")
    rng = np.random.default_rng(9)
    T, E, K, step = 3, 10, 4, 2.0 ** -6
    g = lm().Gating(score=score, renorm=renorm)
    lg = np.round(rng.standard_normal((T, E)) * 64) / 64
    lg = lg.astype(np.float32)
    dg = rng.standard_normal((T, K)).astype(np.float32)
    idx, _ = lm().select(put(lg), None, K, g)
    # the picks kept by a bias that lifts them, in their order
    got = f64(lm().select_backward(put(lg), idx, put(dg), g))
    pick = to_np(idx)
    for t in range(T):
        b = np.zeros(E, np.float32)
        b[pick[t]] = 8 + 4.0 * np.arange(K, 0, -1)
        for e in range(E):
            loss = []
            for sgn in (1, -1):
                moved = lg[t:t + 1].copy()
                moved[0, e] += sgn * step
                i, gate = lm().select(put(moved), put(b), K, g)
                assert (to_np(i)[0] == pick[t]).all()
                loss.append(float((f64(gate)[0] * dg[t]).sum()))
            diff = (loss[0] - loss[1]) / (2 * step)
            bound = np.abs(dg[t]).sum() * (step ** 2 / 6 + 32 * U / step)
            assert abs(diff - got[t, e]) <= bound, (t, e, diff, got[t, e])


# ---- norms ------------------------------------------------------------------------------------

NORMS = [dict(T=1, d=8), dict(T=3, d=64, gate="channel"), dict(T=130, d=6144, post=True, gate="channel"),
         dict(T=33, d=1032, post=True, gate="token"), dict(T=9, d=16384, post=True, gate="channel"),
         dict(T=5, d=8200, gate="token"), dict(T=700, d=520, post=True), dict(T=1100, d=2048, post=True, gate="channel"),
         dict(T=3000, d=128, post=True, gate="token"), dict(T=4, d=12296, noy=True), dict(T=66, d=256, noy=True),
         dict(T=600, d=8200, post=True, gate="channel"), dict(T=530, d=6144, post=True, gate="token"),
         dict(T=515, d=5128, gate="channel"), dict(T=300, d=16384, post=True, gate="token")]


def norm_inputs(kw, dt, seed=4):
    rng = np.random.default_rng(seed)
    T, d = kw["T"], kw["d"]
    if dt == "f32" and d == 1032:
        d = 1028
    rows = lambda s: stored(s * rng.standard_normal((T, d)) * np.exp(0.5 * rng.standard_normal((T, 1))), dt)  # noqa: E731
    c = dict(x=rows(1.0), y=None if kw.get("noy") else rows(2.0), h=rows(1.5), dh=rows(0.01), dz=rows(0.01))
    c["w_pre"] = stored(1 + 0.2 * rng.standard_normal(d), "f32")
    c["w_post"] = stored(1 + 0.2 * rng.standard_normal(d), "f32") if kw.get("post") else None
    gate = {"channel": lambda: 0.5 + 0.2 * rng.standard_normal(d), "token": lambda: rng.random((T, 1)), None: lambda: None}
    g = gate[kw.get("gate")]()
    c["gate"] = None if g is None else stored(g, "f32")
    return c


def pair(c, k, i):
    return None if c[k] is None else c[k][i]


A, B, EPS = 0.875, 0.5, float(np.float32(1e-6))
ROW = 60  # chain of a row's sum


def norm_args(c, i):
    return dict(y=pair(c, "y", i), w_post=pair(c, "w_post", i), gate=pair(c, "gate", i))


def check_norm(c, dt, h, z, a=A, b=B):
    o = norm_args(c, 1)
    rh, rz = ob.block_norm(c["x"][1], o["y"], o["gate"], o["w_post"], c["w_pre"][1], a, b, EPS)
    term = np.abs(rh - a * c["x"][1])
    eh = (ROW / 2 + 8) * U * (np.abs(a * c["x"][1]) + term)  # before the rounding
    if h is not None:
        over = np.abs(f64(h) - rh) - eh * (1 + HALF[dt]) - HALF[dt] * np.abs(rh)
        assert over.max() <= 1e-37, over.max()
    if z is None:
        return
    r = ob.rms(rh, EPS)
    rel = np.sqrt((eh ** 2).sum(1, keepdims=True)) / np.sqrt((rh ** 2).sum(1, keepdims=True) + 1e-300) + (ROW / 2 + 8) * U
    ez = eh * r * np.abs(c["w_pre"][1]) + rel * np.abs(rz)
    over = np.abs(f64(z) - rz) - ez * (1 + HALF[dt]) - HALF[dt] * np.abs(rz)
    assert over.max() <= 1e-37, over.max()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kw", NORMS, ids=lambda k: "_".join(f"{a}{v}" for a, v in k.items()))
def test_block_norm(kw, dt):
    import torch
    say(f"norm {kw} {dt}")
    c = norm_inputs(kw, dt)
    run = lambda: lm().block_norm(c["x"][0], c["w_pre"][0], residual_scale=A, block_scale=B, eps=EPS, **norm_args(c, 0))  # noqa: E731
    h, z = run()
    check_norm(c, dt, h, z)
    h2, z2 = run()
    assert torch.equal(h, h2) and torch.equal(z, z2)


def test_block_norm_forms():
    """No norm before, no residual scale, zeros, and outputs over inputs."""
    import torch
    say("norm forms")
    c = norm_inputs(dict(T=40, d=512, post=True, gate="token"), "bf16")
    x, w = c["x"][0], c["w_pre"][0]
    h, z = lm().block_norm(x, w, eps=EPS)
    assert h is None
    check_norm(dict(c, y=None, gate=None, w_post=None), "bf16", None, z, a=1.0)
    h, z = lm().block_norm(x, None, eps=EPS, residual_scale=A, block_scale=B, **norm_args(c, 0))
    assert z is None
    check_norm(c, "bf16", h, None)
    zero = torch.zeros_like(x)
    h, z = lm().block_norm(zero, w, y=zero, w_post=w, eps=EPS)
    assert not h.any() and not z.any()
    from mixture_experts_layer_router_amd import block as lb
    n = lb.Norm(A, B, EPS, lb.GATE_TOKEN)
    ref = lm().block_norm(x, w, residual_scale=A, block_scale=B, eps=EPS, **norm_args(c, 0))
    x2, y2 = x.clone(), c["y"][0].clone()
    lb.lc_moe_block_norm(40, 512, lm().BF16, n, x2, y2, c["gate"][0], c["w_post"][0], w, x2, y2)
    assert torch.equal(x2, ref[0]) and torch.equal(y2, ref[1])


def check_norm_backward(c, dt, out, T, d, wgs):
    o = norm_args(c, 1)
    ref = ob.block_norm_backward(c["h"][1], pair(c, "dh", 1), pair(c, "dz", 1), o["y"], o["gate"], o["w_post"],
                                 c["w_pre"][1], A, B, EPS)
    chain = T / wgs + 3 + wgs / 16 + 18
    for k in ("dx", "dy", "dw_pre", "dw_post", "dgate"):
        assert (k in out) == (k in ref), k
        if k not in ref:
            continue
        if k in ("dx", "dy"):
            C, half = 4 * ROW, HALF[dt]
        else:
            C, half = 4 * ROW + chain, 0.0
        over = np.abs(f64(out[k]) - ref[k]) - C * U * (1 + half) * ref[k + "_mag"] - half * np.abs(ref[k])
        assert over.max() <= 1e-37, (k, over.max())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kw", NORMS, ids=lambda k: "_".join(f"{a}{v}" for a, v in k.items()))
def test_block_norm_backward(kw, dt):
    import torch
    from mixture_experts_layer_router_amd import block as lb
    say(f"norm backward {kw} {dt}")
    c = norm_inputs(kw, dt)
    T, d = c["h"][0].shape
    run = lambda: lm().block_norm_backward(c["h"][0], c["w_pre"][0], c["dz"][0], dh=c["dh"][0], residual_scale=A,  # noqa: E731
                                           block_scale=B, eps=EPS, **norm_args(c, 0))
    out = run()
    wgs = lb.lc_moe_block_norm_backward_workspace_size(T, d, lm().BF16 if dt == "bf16" else lm().F32) // (12 * d)
    check_norm_backward(c, dt, out, T, d, max(wgs, 1))
    again = run()
    for k in out:
        assert torch.equal(out[k], again[k]), k


def test_block_norm_backward_forms():
    """No dh, no dz, no rows, and outputs over inputs."""
    import torch
    from mixture_experts_layer_router_amd import block as lb
    say("norm backward forms")
    c = norm_inputs(dict(T=50, d=264, post=True, gate="channel"), "bf16")
    kw = dict(residual_scale=A, block_scale=B, eps=EPS, **norm_args(c, 0))
    out = lm().block_norm_backward(c["h"][0], c["w_pre"][0], c["dz"][0], **kw)
    check_norm_backward(dict(c, dh=None), "bf16", out, 50, 264, 50)
    out = lm().block_norm_backward(c["h"][0], c["w_pre"][0], None, dh=c["dh"][0], **kw)
    assert not out["dw_pre"].any()
    check_norm_backward(dict(c, dz=None), "bf16", out, 50, 264, 50)
    ref = lm().block_norm_backward(c["h"][0], c["w_pre"][0], c["dz"][0], dh=c["dh"][0], **kw)
    n = lb.Norm(A, B, EPS, lb.GATE_CHANNEL)
    dh, y = c["dh"][0].clone(), c["y"][0].clone()
    s = [torch.empty(264, device=device()) for _ in range(3)]
    ws = torch.empty(lb.lc_moe_block_norm_backward_workspace_size(50, 264, 1), dtype=torch.uint8, device=device())
    lb.lc_moe_block_norm_backward(50, 264, 1, n, c["h"][0], dh, c["dz"][0], y, c["gate"][0], c["w_post"][0], c["w_pre"][0],
                                  dh, y, *s, ws)
    assert torch.equal(dh, ref["dx"]) and torch.equal(y, ref["dy"])
    for k, t in zip(("dw_pre", "dw_post", "dgate"), s):
        assert torch.equal(ref[k], t), k
    e = torch.empty((0, 264), dtype=torch.bfloat16, device=device())
    out = lm().block_norm_backward(e, c["w_pre"][0], e, y=e, w_post=c["w_post"][0], gate=c["gate"][0])
    assert out["dx"].shape == (0, 264) and not out["dw_pre"].any() and not out["dw_post"].any() and not out["dgate"].any()


# ---- block FP8 --------------------------------------------------------------------------------

def fp8_parts(buf, R, C):
    """(codes [R][Cp], exponents k [R][Cp/128], the scale bytes of rows that are none)."""
    raw = to_np(buf)
    cp, rp = -(-C // 128) * 128, -(-R // 256) * 256
    codes = raw[:R * cp].reshape(R, cp)
    at = -(-R * cp // 256) * 256
    sc = raw[at:at + cp // 128 * rp].reshape(cp // 128, rp)
    r = np.arange(rp)
    place = (r & ~127) + 4 * (r & 31) + (r >> 5 & 3)
    sc = sc[:, place].T.astype(int) - 127
    return codes, sc[:R], sc[R:], raw[at + cp // 128 * rp:]


def check_matrix(buf, codes, k, rows):
    """Against codes and exponents of blocks of rows x 128."""
    R, C = codes.shape
    c, s, rest, tail = fp8_parts(buf, R, C)
    np.testing.assert_array_equal(c[:, :C], codes)
    assert not c[:, C:].any()
    np.testing.assert_array_equal(s, k.repeat(rows, 0)[:R])
    assert not rest.any() and (tail == 127).all()


QM = [(1, 8), (1, 200), (3, 128), (64, 136), (128, 128), (130, 520), (257, 256), (300, 1032), (511, 64)]


@pytest.mark.parametrize("R,C", QM)
@pytest.mark.parametrize("block", [1, 128])
def test_quantize_matrix(R, C, block):
    say(f"quantize {R}x{C} block {block}")
    rng = np.random.default_rng(R * 7 + C)
    v = rng.standard_normal((R, C)) * np.exp2(rng.integers(-20, 20, (R, C)) * (rng.random((R, C)) < 0.3))
    v[0, :min(C, 70)] = 0.0
    x, xv = stored(v, "bf16")
    m = lm().quantize_matrix(x, block_rows=block, transposed=True)
    one = lm().quantize_matrix(x, block_rows=block)
    t = lm().quantize_matrix(x, block_rows=block, rows=False, transposed=True)
    assert t.data is None and one.t is None
    for buf, values in ((m.data, xv), (one.data, xv), (m.t, xv.T), (t.t, xv.T)):
        codes, k = ob.quantize(values, block, 128)
        check_matrix(buf, codes, k, block)


def test_quantize_every_bf16_value():
    """Every bf16 value up to its block's 448, each in the last 64 places of a block whose largest is
    448 * 2^k: ties, subnormal codes and signs."""
    import torch
    say("quantize every value")
    bits = torch.arange(65536, dtype=torch.int32)
    vals = (bits << 16).view(torch.float32)
    ok = torch.isfinite(vals) & (vals.abs() <= 448)
    vals = vals[ok]
    n = -(-len(vals) // 64) * 64
    v = torch.zeros(n)
    v[:len(vals)] = vals
    x = torch.cat((torch.full((n // 64, 64), 448.0), v.view(-1, 64)), 1)
    x[0, 0] = 448.0
    xb = x.to(torch.bfloat16)
    m = lm().quantize_matrix(xb.to(device()), block_rows=1, transposed=False)
    codes, k = ob.quantize(xb.double().numpy(), 1, 128)
    assert not k.any()
    check_matrix(m.data, codes, k, 1)
    # blocks of tiny values: the scale ends at 2^-127
    tiny = (torch.arange(256, dtype=torch.int32) << 16).view(torch.float32).view(2, 128).to(torch.bfloat16)
    m = lm().quantize_matrix(tiny.to(device()), block_rows=1)
    check_matrix(m.data, *ob.quantize(tiny.double().numpy(), 1, 128), 1)


def product(a, b, add=None):
    """(A B^T + add, bound of its error before the rounding)."""
    c = a @ b.T
    rss = np.sqrt((a * a) @ (b * b).T)
    err = 2.0 ** -11 * (np.abs(c) + rss)
    return (c if add is None else c + add), err + (0 if add is None else U * np.abs(add))


def check_product(got, c, err):
    over = np.abs(f64(got) - c) - err * (1 + HALF["bf16"]) - HALF["bf16"] * np.abs(c)
    assert over.max() <= 1e-37, over.max()


MM = [(1, 8, 8), (1, 136, 128), (5, 64, 200), (64, 520, 1032), (130, 128, 384), (128, 264, 640), (257, 512, 136),
      (300, 776, 520), (33, 2048, 3328), (1000, 1000, 256), (2100, 6152, 264), (4096, 3200, 128)]


@pytest.mark.parametrize("M,N,K", MM)
@pytest.mark.parametrize("add", [False, True])
def test_matmul(M, N, K, add):
    import torch
    say(f"matmul {M} {N} {K} add {add}")
    rng = np.random.default_rng(M + N + K)
    grow = lambda n: np.exp2(rng.integers(-6, 7, (n, 1)))  # noqa: E731
    a, av = stored(rng.standard_normal((M, K)) * grow(M), "bf16")
    b, bv = stored(rng.standard_normal((N, K)) / np.sqrt(K), "bf16")
    e, ev = stored(rng.standard_normal((M, N)), "bf16") if add else (None, None)
    am, bm = lm().quantize_matrix(a, block_rows=1), lm().quantize_matrix(b)
    got = lm().matmul_fp8(am, bm, add=e)
    c, err = product(ob.quantized(av, 1, 128), ob.quantized(bv, 128, 128), ev)
    check_product(got, c, err)
    assert torch.equal(got, lm().matmul_fp8(am, bm, add=e))
    if add:  # over the addend itself
        e2 = e.clone()
        assert lm().matmul_fp8(am, bm, add=e2, out=e2) is e2 and torch.equal(e2, got)


@pytest.mark.parametrize("T,k,n", [(1, 136, 264), (17, 520, 8), (64, 1024, 1032), (200, 256, 384), (777, 1032, 520),
                                   (2100, 1032, 1032), (1030, 2056, 2048)])
def test_linear(T, k, n):
    import torch
    say(f"linear {T} {k} {n}")
    rng = np.random.default_rng(T + k + n)
    x, xv = stored(rng.standard_normal((T, k)) * np.exp2(rng.integers(-4, 5, (T, 1))), "bf16")
    w, wv = stored(rng.standard_normal((n, k)) / np.sqrt(k), "bf16")
    dy, dv = stored(1e-3 * rng.standard_normal((T, n)), "bf16")
    da, dav = stored(1e-3 * rng.standard_normal((T, k)), "bf16")
    wq = lm().quantize_matrix(w, transposed=True)
    q = ob.quantized(wv, 128, 128)
    y = lm().linear_fp8(x, wq)
    check_product(y, *product(ob.quantized(xv, 1, 128), q))
    if T * n * k > 2e9:  # smaller products may be summed up in another order
        assert torch.equal(y, lm().matmul_fp8(lm().quantize_matrix(x, block_rows=1), wq))
    out = lm().linear_fp8_backward(dy, x, wq)
    check_product(out["dx"], *product(ob.quantized(dv, 1, 128), q.T))
    check_product(out["dw"], *product(ob.quantized(dv.T, 1, 128), ob.quantized(xv.T, 1, 128)))
    over = da.clone()
    r = lm().linear_fp8_backward(dy, x, wq, dx_add=over, dx=over, need_dw=False)
    assert "dw" not in r and r["dx"] is over
    check_product(over, *product(ob.quantized(dv, 1, 128), q.T, dav))
    r = lm().linear_fp8_backward(dy, x, wq, need_dx=False)
    assert "dx" not in r and torch.equal(r["dw"], out["dw"])


FEW = [(1, 8, 8), (1, 128, 40), (3, 1032, 72), (15, 2048, 264), (16, 6144, 136), (17, 264, 1032), (32, 4104, 24),
       (33, 136, 520), (63, 2056, 40), (64, 16384, 8), (65, 1032, 72), (64, 2048, 6144), (64, 2048, 5344),
       (100, 64, 64), (400, 520, 520), (777, 1032, 520), (1600, 72, 40), (4000, 64, 64), (200, 6144, 136), (777, 520, 520)]


@pytest.mark.parametrize("T,k,n", FEW)
def test_linear_few_tokens(T, k, n):
    """Few tokens: around the blocks of 16 of them, odd runs, reductions split and not; the addend, and the
    same workspace for both."""
    import torch
    say(f"linear of few tokens {T} {k} {n}")
    rng = np.random.default_rng(T + k + n)
    x, xv = stored(rng.standard_normal((T, k)) * np.exp2(rng.integers(-8, 9, (T, 1))), "bf16")
    w, wv = stored(rng.standard_normal((n, k)) / np.sqrt(k) * np.exp2(rng.integers(-3, 4, (n, 1))), "bf16")
    e, ev = stored(rng.standard_normal((T, n)), "bf16")
    wq, qx, qw = lm().quantize_matrix(w), ob.quantized(xv, 1, 128), ob.quantized(wv, 128, 128)
    y = lm().linear_fp8(x, wq)
    check_product(y, *product(qx, qw))
    assert torch.equal(y, lm().linear_fp8(x, wq))
    over = e.clone()
    assert lm().linear_fp8(x, wq, add=over, out=over) is over
    check_product(over, *product(qx, qw, ev))
    assert torch.equal(over, lm().linear_fp8(x, wq, add=e))
    # a token's result does not depend on the others
    if T > 1:
        assert torch.equal(lm().linear_fp8(torch.cat((x[1:], x[:1])), wq), torch.cat((y[1:], y[:1])))


def test_linear_few_tokens_every_bf16_value():
    """One-hot weights give the tokens' codes themselves: every finite bf16 value up to its run's 448, and the
    values of the smallest scale."""
    import torch
    say("linear of every value")
    vals = (torch.arange(65536, dtype=torch.int32) << 16).view(torch.float32)
    vals = vals[torch.isfinite(vals) & (vals.abs() <= 448)]
    n = -(-len(vals) // 64) * 64
    v = torch.zeros(n)
    v[:len(vals)] = vals
    x = torch.cat((torch.full((n // 64, 64), 448.0), v.view(-1, 64)), 1).to(torch.bfloat16)
    tiny = (torch.arange(256, dtype=torch.int32) << 16).view(torch.float32).view(2, 128).to(torch.bfloat16)
    big = (torch.arange(0x7F00, 0x7F80, dtype=torch.int32) << 16).view(torch.float32).view(1, 128).to(torch.bfloat16)
    for rows, unit in ((x, 1.0), (tiny, 2.0 ** 120), (big, 2.0 ** -20), (-big, 2.0 ** -20)):
        wq = lm().quantize_matrix((unit * torch.eye(128)).to(torch.bfloat16).to(device()))
        want = torch.from_numpy(ob.quantized(rows.double().numpy(), 1, 128) * unit)
        for i in range(0, len(rows), 64):
            got = lm().linear_fp8(rows[i:i + 64].to(device()), wq).double().cpu()
            assert torch.equal(got, want[i:i + 64]), (i, unit)


def test_linear_few_tokens_refuses_its_input_as_output():
    import torch
    say("linear over its input")
    x = put(np.ones((4, 16), np.float32), torch.bfloat16)
    wq = lm().quantize_matrix(put(np.ones((16, 16), np.float32), torch.bfloat16))
    with pytest.raises(Exception):
        lm().linear_fp8(x, wq, out=x)


def test_no_rows():
    import torch
    say("no rows")
    w = put(np.ones((16, 24), np.float32), torch.bfloat16)
    wq = lm().quantize_matrix(w, transposed=True)
    x = torch.empty((0, 24), dtype=torch.bfloat16, device=device())
    assert lm().linear_fp8(x, wq).shape == (0, 16)
    out = lm().linear_fp8_backward(torch.empty((0, 16), dtype=torch.bfloat16, device=device()), x, wq)
    assert out["dx"].shape == (0, 24) and not out["dw"].any()
    h, z = lm().block_norm(x, torch.ones(24, device=device()), y=x)
    assert h.shape == z.shape == (0, 24)
