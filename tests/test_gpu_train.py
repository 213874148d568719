"""GPU parity of the training operators against the fp64 oracle (oracle/train.py).

Tolerances.  u = 2^-24 is half an fp32 step relative to the value, 2^-8 half a bf16 one.
  * A probability is exp(l - m) / sum: l - m is rounded once (|l - m| u absolute in the
    exponent), exp, the sum of at most 64 terms a lane and 6 across lanes, the reciprocal and
    the product add a few u each, so |dp| <= (|l - m| + 80) u p; the logits here have
    |l - m| <= 24: 128 u p covers it.
  * A dot product of n fp32 terms added along chains of c terms is off by at most
    (c + 2) u sum |a b|.
  * Products split into bf16 parts: the parts that are left out are at most 4 u of a
    product for 24-bit parts and 2^-16 of it for the 16-bit parts of a bf16 dx, which is
    rounded to bf16 besides.  Operands rounded to fp16 (a bf16 dx of many tokens) are off by
    2^-11 each, a product by 2^-10 (1 + 2^-12); below 2^-14 of fp16, which is 2^-28 of the
    row's largest value here, by 2^-25 of fp16 = 2^-39 of that largest value.
Each bound below is such a sum; none is fitted to a result.
"""
import numpy as np
import pytest

from gpu_common import device, rel_l2, say, to_np
from oracle import train as ot

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def bf16_round(a):
    import torch
    return torch.tensor(np.asarray(a, np.float32)).to(torch.bfloat16)


def put(a, dtype=None):
    import torch
    t = torch.tensor(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(device())


def pick(rng, T, E, K):
    return np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)


# ---- balance loss ---------------------------------------------------------------------------

BAL = [dict(T=1, E=1, K=1), dict(T=1, E=7, K=3), dict(T=64, E=96, K=6), dict(T=65, E=97, K=2, off=[0, 1, 1, 40, 65]),
       dict(T=300, E=260, K=12, off=[3, 64, 64, 128, 129, 280], pad=0.4), dict(T=128, E=64, K=8, off=list(range(129))),
       dict(T=1000, E=768, K=12, off=[0, 0, 999, 1000, 1000], pad=0.1), dict(T=257, E=1029, K=5, pad=0.5),
       dict(T=70, E=4096, K=16, off=[0, 35, 70]), dict(T=130, E=2050, K=1),
       dict(T=40, E=12, K=12, off=[0, 20, 40]), dict(T=50, E=8, K=2, pad=1.0)]


def balance_inputs(kw, seed=1):
    T, E, K = kw["T"], kw["E"], kw["K"]
    rng = np.random.default_rng(seed)
    lg = np.clip(2 * rng.standard_normal((T, E)), -8, 8).astype(np.float32)
    mask = (rng.random(T) >= kw["pad"]).astype(np.uint8) if "pad" in kw else None
    off = np.array(kw["off"], np.int32) if "off" in kw else None
    return lg, pick(rng, T, E, K), off, mask


def run_balance(lg, idx, off, mask, a, z, N=None, **kw):
    import mixture_experts_layer_router_amd as lm
    E = lg.shape[1]
    return lm.balance_loss(put(lg), put(idx), N or min(E, 2048), a, z, None if off is None else put(off),
                           None if mask is None else put(mask), **kw)


def check_balance(r, ref, a, z, T):
    E = ref["p"].shape[1]
    np.testing.assert_array_equal(to_np(r["load"]), ref["load"])
    # a sum over a sequence's tokens: 16 along a wave, 4 waves, a quarter of the blocks, 4
    chain = 16 + 4 + (T // 64 + 2) / 4 + 4
    np.testing.assert_allclose(to_np(r["prob"]), ref["prob"], rtol=(128 + chain) * U, atol=1e-37)
    np.testing.assert_allclose(to_np(r["loss"]), ref["loss"], rtol=(256 + chain + 64) * U, atol=1e-37)
    # |d| <= p (|u| + sum p |u| + |zl|) (2 probabilities, 70 additions, a few products)
    seq, p = ref["seq"], ref["p"]
    live = max((ref["n"] > 0).sum(), 1)
    mag = np.zeros_like(p)
    for s, n in enumerate(ref["n"]):
        if n:
            K = idx_K(ref)
            c = abs(a) / (live * n) * np.abs(E * ref["load"][s] / (K * n) - 1)
            rows = seq == s
            mag[rows] = p[rows] * (c + (p[rows] * c).sum(1, keepdims=True))
    lse = ot.softmax(ref["logits"])[1]
    total = max(ref["n"].sum(), 1)
    mag += np.where(seq[:, None] >= 0, p * (2 * abs(z) / total * np.abs(np.where(np.isfinite(lse), lse, 0)))[:, None], 0)
    got = to_np(r["dlogits"]).astype(np.float64)
    assert not got[seq < 0].any()
    over = np.abs(got - ref["dlogits"]) - (2 * 128 + 80) * U * mag
    assert over.max() <= 1e-37, over.max()


def idx_K(ref):
    return ref["idx"].shape[1]


def reference(lg, idx, off, mask, a, z):
    ref = ot.balance_loss(lg, idx, a, z, off, mask)
    ref["idx"] = idx
    keep = np.ones(lg.shape[0], bool) if mask is None else mask != 0
    ref["logits"] = np.where(keep[:, None], lg, 0.0)
    return ref


@pytest.mark.parametrize("kw", BAL, ids=lambda k: f"T{k['T']}_E{k['E']}_K{k['K']}_S{len(k.get('off', [0, 0])) - 1}")
@pytest.mark.parametrize("a,z", [(0.01, 0.0), (0.5, 1e-3)])
def test_balance(kw, a, z):
    import torch
    say(f"balance {kw} a={a} z={z}")
    lg, idx, off, mask = balance_inputs(kw)
    a, z = float(np.float32(a)), float(np.float32(z))
    ref = reference(lg, idx, off, mask, a, z)
    r = run_balance(lg, idx, off, mask, a, z)
    check_balance(r, ref, a, z, kw["T"])
    again = run_balance(lg, idx, off, mask, a, z)
    for k in r:
        assert torch.equal(r[k], again[k]), k


@pytest.mark.parametrize("T,S,kind", [(1500, 1500, "one"), (900, 4000, "sparse"), (900, 65535, "sparse"),
                                      (2000, 63, "even"), (2000, 64, "even"), (2000, 129, "even"), (600, 300, "late")])
def test_balance_many_sequences(T, S, kind):
    """More sequences than a wave has lanes: of one token each, mostly empty ones, as many as
    fill the lanes, and tokens in front of the first and behind the last."""
    say(f"balance T={T} S={S} {kind}")
    rng = np.random.default_rng(S)
    E, K = 12, 3
    lg = rng.standard_normal((T, E)).astype(np.float32)
    idx = rng.integers(0, E, (T, K)).astype(np.int32)
    if kind in ("one", "even"):
        off = np.linspace(0, T, S + 1).astype(np.int32)
    elif kind == "sparse":
        off = np.sort(rng.choice(np.arange(0, T + 1, 7), S + 1)).astype(np.int32)
    else:
        off = np.linspace(400, 580, S + 1).astype(np.int32)
    ref = reference(lg, idx, off, None, 0.5, float(np.float32(1e-3)))
    check_balance(run_balance(lg, idx, off, None, 0.5, float(np.float32(1e-3))), ref, 0.5, float(np.float32(1e-3)), T)


def test_balance_masked_rows_may_hold_anything():
    """NaN and infinities in rows that the mask or the offsets leave out, picks out of range,
    logits of -infinity and of the lowest value, a row of nothing but -infinity."""
    import torch
    T, E, K = 90, 50, 4
    rng = np.random.default_rng(5)
    lg = rng.standard_normal((T, E)).astype(np.float32)
    idx = pick(rng, T, E, K)
    idx[5, 0], idx[6, 1], idx[7] = -1, E, [3, 3, 3, 3]
    off, mask = np.array([4, 30, 80], np.int32), (rng.random(T) > 0.3).astype(np.uint8)
    mask[[10, 11, 12, 13, 40]] = [0, 1, 1, 1, 1]
    lg[mask == 0] = np.nan
    lg[:4], lg[80:] = np.inf, np.nan
    lg[11] = -np.inf
    lg[12, :25] = -np.inf
    lg[13] = np.finfo(np.float32).min
    lg[40, 7:] = np.finfo(np.float32).min
    say("balance with masked rows")
    ref = reference(lg, idx, off, mask, 0.1, 0.0)
    assert ref["seq"][11] == -1
    r = run_balance(lg, idx, off, mask, 0.1, 0.0)
    check_balance(r, ref, 0.1, 0.0, T)
    assert bool(torch.isfinite(r["dlogits"]).all()) and bool(torch.isfinite(r["loss"]).all())


def test_balance_even_load_gives_exactly_zero():
    T, E, K = 96, 12, 3
    idx = ((np.arange(T)[:, None] * K + np.arange(K)) % E).astype(np.int32)
    lg = np.random.default_rng(6).standard_normal((T, E)).astype(np.float32)
    r = run_balance(lg, idx, None, None, 0.3, 0.0)
    assert not bool(r["dlogits"].any())
    # loss = a * sum of the mean probabilities = a, within the probabilities' own error
    assert abs(float(r["loss"][0]) - float(np.float32(0.3))) <= 0.3 * 256 * U


def test_balance_offsets_out_of_range_are_clamped():
    lg, idx, _, _ = balance_inputs(dict(T=50, E=20, K=3))
    off = np.array([-5, 20, 99], np.int32)
    r = run_balance(lg, idx, off, None, 0.1, 0.01)
    check_balance(r, reference(lg, idx, np.array([0, 20, 50]), None, float(np.float32(0.1)), float(np.float32(0.01))),
                  0.1, 0.01, 50)


@pytest.mark.parametrize("T,E", [(50, 20), (300, 70), (90, 600)])
def test_balance_descending_offsets_stay_in_range(T, E):
    """Unspecified numbers, but every output is written in place: the rows around them keep
    their values, and the next call is right."""
    import torch
    from mixture_experts_layer_router_amd import train as lt
    import mixture_experts_layer_router_amd as lm
    lg, idx, _, _ = balance_inputs(dict(T=T, E=E, K=3))
    dev, S = device(), 4
    shape = lm.make_shape(T, 8, E, 0, 3, 8, lm.BF16)
    ws = torch.zeros(lt.lc_moe_balance_workspace_size(shape, S), dtype=torch.uint8, device=dev)
    for off in ([T // 2, 0, T, 3, T // 3], [T, T // 2, 5, 1, 0], [0, T, 0, T, 0]):
        dl = torch.full((T + 8, E), 7.0, device=dev)
        load = torch.full((S + 8, E), 7, dtype=torch.int32, device=dev)
        prob = torch.full((S + 8, E), 7.0, device=dev)
        loss = torch.full((4,), 7.0, device=dev)
        lt.lc_moe_balance_loss(shape, lt.BalanceCoef(0.1, 0.1), put(lg), put(idx), put(np.array(off, np.int32)), S, None, loss,
                               load, prob, dl, ws)
        torch.cuda.synchronize()
        assert bool((dl[T:] == 7).all()) and bool((load[S:] == 7).all()) and bool((prob[S:] == 7).all())
        assert bool((loss[2:] == 7).all()) and not bool((dl[:T] == 7).any())
    good = np.array([0, 5, T // 2, T // 2, T], np.int32)
    r = run_balance(lg, idx, good, None, 0.1, 0.1)
    check_balance(r, reference(lg, idx, good, None, float(np.float32(0.1)), float(np.float32(0.1))), 0.1, 0.1, T)


def test_balance_without_gradient():
    import torch
    lg, idx, off, mask = balance_inputs(BAL[4])
    a, b = run_balance(lg, idx, off, mask, 0.1, 0.01), run_balance(lg, idx, off, mask, 0.1, 0.01, need_grad=False)
    assert b["dlogits"] is None
    for k in ("loss", "load", "prob"):
        assert torch.equal(a[k], b[k])


# ---- gate gradient --------------------------------------------------------------------------

GATE = [dict(T=1, d=8, K=1), dict(T=1, d=4, K=3, f32=True), dict(T=7, d=72, K=5), dict(T=33, d=1028, K=6, f32=True),
        dict(T=64, d=6144, K=12), dict(T=100, d=520, K=8), dict(T=5, d=16392, K=2), dict(T=300, d=64, K=33),
        dict(T=3, d=40000, K=2, f32=True)]


@pytest.mark.parametrize("kw", GATE, ids=lambda k: f"T{k['T']}_d{k['d']}_K{k['K']}_{'f32' if k.get('f32') else 'bf16'}")
def test_gate_backward(kw):
    import torch
    import mixture_experts_layer_router_amd as lm
    say(f"gate {kw}")
    T, d, K = kw["T"], kw["d"], kw["K"]
    rng = np.random.default_rng(T + d)
    dt = torch.float32 if kw.get("f32") else torch.bfloat16
    # every row in use once, some picks zero-computation, one row index past the rows
    ffn = rng.random((T, K)) < 0.7
    slot = np.full((T, K), -1, np.int32)
    slot[ffn] = rng.permutation(int(ffn.sum()))
    R = max(int(ffn.sum()), 1)
    if T > 1:
        slot[0, 0] = R + 7
    t = [put(rng.standard_normal(s), dt) for s in ((T, d), (R, d), (T, d))]
    x, rows, dy = (to_np(v).astype(np.float64) for v in t)
    got = lm.gate_backward(t[0], t[1], put(slot), t[2])
    ref, mag = ot.gate_backward(x, rows, slot, dy)
    chain = d / 64 + 16
    over = np.abs(to_np(got) - ref) - (chain + 2) * U * mag
    assert over.max() <= 0, over.max()
    assert torch.equal(got, lm.gate_backward(t[0], t[1], put(slot), t[2]))


def test_gate_backward_without_rows():
    """No FFN pick at all: num_rows = 0."""
    import torch
    import mixture_experts_layer_router_amd as lm
    x = torch.ones(4, 16, device=device())
    got = lm.gate_backward(x, torch.empty(0, 16, device=device()), torch.full((4, 3), -1, dtype=torch.int32, device=device()),
                           2 * x)
    assert bool((got == 32).all())


# ---- router backward ------------------------------------------------------------------------

ROUTER = [dict(T=1, d=8, E=1, K=1), dict(T=1, d=4, E=5, K=2, f32=True), dict(T=3, d=64, E=12, K=3),
          dict(T=64, d=256, E=96, K=6, aux=True, add=True), dict(T=77, d=1028, E=77, K=5, f32=True),
          dict(T=300, d=520, E=33, K=4, aux=True), dict(T=513, d=328, E=257, K=7, add=True),
          dict(T=200, d=132, E=300, K=3, f32=True, aux=True, add=True), dict(T=40, d=64, E=4096, K=9, aux=True),
          dict(T=30, d=36, E=2050, K=2, f32=True), dict(T=1500, d=72, E=40, K=2), dict(T=2100, d=320, E=768, K=12),
          dict(T=64, d=1040, E=768, K=12, aux=True, add=True), dict(T=65, d=24, E=160, K=3, f32=True, add=True),
          dict(T=33, d=88, E=45, K=3, f32=True, aux=True, add=True),
          # many tokens: fp16 operands (with and without dx_add), fp32's big tiles, ragged edges
          dict(T=1100, d=13320, E=140, K=4, aux=True, add=True), dict(T=4111, d=4104, E=133, K=3, aux=True),
          dict(T=1030, d=6700, E=130, K=2, f32=True, aux=True, add=True)]


def router_inputs(kw, seed=3):
    import torch
    T, d, E, K = kw["T"], kw["d"], kw["E"], kw["K"]
    rng = np.random.default_rng(seed)
    dt = torch.float32 if kw.get("f32") else torch.bfloat16
    x = put(rng.standard_normal((T, d)), dt)
    w = put((rng.standard_normal((E, d)) / np.sqrt(d)).astype(np.float32))
    lg = put(np.clip(1.5 * rng.standard_normal((T, E)), -8, 8).astype(np.float32))
    idx = put(pick(rng, T, E, K))
    dg = put(rng.standard_normal((T, K)).astype(np.float32))
    aux = put((0.01 * rng.standard_normal((T, E))).astype(np.float32)) if kw.get("aux") else None
    add = put(0.1 * rng.standard_normal((T, d)), dt) if kw.get("add") else None
    return x, w, lg, idx, dg, aux, add


def check_router(r, x, w, lg, idx, dg, aux, add):
    import torch
    f = lambda t: None if t is None else to_np(t).astype(np.float64)  # noqa: E731
    i = to_np(idx)
    xs, ws, au, ad = f(x), f(w), f(aux), f(add)
    T, d = xs.shape
    E = ws.shape[0]
    ref = ot.router_backward(xs, ws, f(lg), i, f(dg), au, ad)
    _, p, dp = ot.dlogits(f(lg), i, f(dg))
    # dlogits: p (|dp| + sum p |dp|) with two probabilities and at most 80 additions, and the sum
    err = (2 * 128 + 80) * U * p * (np.abs(dp) + (p * np.abs(dp)).sum(1, keepdims=True))
    if au is not None:
        err = err + U * np.abs(ref["dlogits"])
    if "dlogits" in r:
        over = np.abs(f(r["dlogits"]) - ref["dlogits"]) - err
        assert over.max() <= 1e-37, over.max()
    half = x.dtype == torch.bfloat16
    mag = np.abs(ref["dlogits"]) @ np.abs(ws)
    # at most three partial products an expert, added in one chain
    f16 = half and T > 64 and -(-T // 128) * -(-d // 256) >= 384
    part = 2.0 ** -10 * (1 + 2.0 ** -11) if f16 else 2.0 ** -16 if half else 4 * U
    tol = err @ np.abs(ws) + ((3 * E + 8) * U + part) * mag
    if f16:  # what falls below fp16's normal numbers in a row of W_r or of 2^wexp dlogits
        top = np.abs(ws).max(1)
        rows = (np.abs(ref["dlogits"]) * top).max(1, keepdims=True)
        tol = tol + 2.0 ** -38 * (np.abs(ref["dlogits"]) @ top)[:, None] + 2.0 ** -38 * E * rows
    if "dx" in r:
        want = ref["dx"]
        tol = tol + (2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8) if half else U * np.abs(want))
        over = np.abs(f(r["dx"]) - want) - tol
        assert over.max() <= 1e-37, over.max()
        # as a whole: one rounding to nearest of independent values is off by about half of its
        # largest error, and fp32 sums by far less than their bound
        assert rel_l2(f(r["dx"]), want) <= (2.0 ** -8 if half else 2e-6)
    if "dw_router" in r:
        want = ref["dw_router"]
        tol = err.T @ np.abs(xs) + ((6 * T + 8) * U + 4 * U) * (np.abs(ref["dlogits"]).T @ np.abs(xs))
        over = np.abs(f(r["dw_router"]) - want) - tol
        assert over.max() <= 1e-37, over.max()
        if E > 1:  # one expert: p = 1, the gradient of the gates is zero and only rounding is left
            assert rel_l2(f(r["dw_router"]), want) <= 5e-6


@pytest.mark.parametrize("kw", ROUTER, ids=lambda k: f"T{k['T']}_d{k['d']}_E{k['E']}_{'f32' if k.get('f32') else 'bf16'}")
def test_router_backward(kw):
    import torch
    import mixture_experts_layer_router_amd as lm
    say(f"router backward {kw}")
    a = router_inputs(kw)
    x, w, lg, idx, dg, aux, add = a
    call = lambda **k: lm.router_backward(x, w, lg, idx, dg, min(kw["E"], 2048), dlogits_aux=aux, dx_add=add, **k)  # noqa: E731
    r = call(need_dlogits=True)
    if kw["E"] > 1:
        check_router(r, *a)
    again = call(need_dlogits=False)
    for k in ("dx", "dw_router"):
        assert torch.equal(r[k], again[k]), k
    # each output alone is the same
    assert torch.equal(call(need_dw=False)["dx"], r["dx"])
    assert torch.equal(call(need_dx=False)["dw_router"], r["dw_router"])


def test_router_backward_aliases():
    """dx written over dx_add, dlogits over dlogits_aux."""
    import torch
    import mixture_experts_layer_router_amd as lm
    from mixture_experts_layer_router_amd import train as lt
    kw = dict(T=150, d=136, E=40, K=4, aux=True, add=True)
    x, w, lg, idx, dg, aux, add = router_inputs(kw)
    r = lm.router_backward(x, w, lg, idx, dg, 30, dlogits_aux=aux, dx_add=add, need_dlogits=True)
    shape = lm.make_shape(150, 136, 30, 10, 4, 8, lm.BF16)
    ws = torch.empty(lt.lc_moe_router_backward_workspace_size(shape), dtype=torch.uint8, device=device())
    dw = torch.empty_like(w)
    lt.lc_moe_router_backward(shape, x, w, lg, idx, dg, aux, add, add, dw, aux, ws)
    assert torch.equal(add, r["dx"]) and torch.equal(aux, r["dlogits"]) and torch.equal(dw, r["dw_router"])


def test_router_backward_of_losses_alone():
    """No gradient from the gates: dlogits = dlogits_aux; neither given: zeros (+ dx_add)."""
    import torch
    import mixture_experts_layer_router_amd as lm
    kw = dict(T=90, d=72, E=20, K=2, aux=True, add=True)
    x, w, lg, idx, dg, aux, add = router_inputs(kw)
    r = lm.router_backward(x, w, None, None, None, 12, dlogits_aux=aux, need_dlogits=True)
    assert torch.equal(r["dlogits"], aux)
    check = to_np(aux).astype(np.float64).T @ to_np(x).astype(np.float64)
    assert rel_l2(to_np(r["dw_router"]), check) <= 5e-6
    r = lm.router_backward(x, w, None, None, None, 12, dx_add=add)
    assert torch.equal(r["dx"], add) and not bool(r["dw_router"].any())


def test_router_backward_odd_picks_and_logits():
    """A repeated pick adds, one out of range does nothing, logits of -infinity are experts that
    cannot be picked, a row of nothing else has no gradient."""
    import mixture_experts_layer_router_amd as lm
    kw = dict(T=20, d=64, E=9, K=3)
    x, w, lg, idx, dg, _, _ = router_inputs(kw)
    idx[0, :], idx[1, 0], idx[2, 1] = 4, -3, 9
    lg[3, 2:] = -np.inf
    idx[3] = put(np.array([0, 1, 0], np.int32))
    lg[4] = -np.inf
    r = lm.router_backward(x, w, lg, idx, dg, 9, need_dlogits=True)
    assert not bool(r["dlogits"][4].any()) and not bool(r["dlogits"][3, 2:].any())
    check_router(r, x, w, lg, idx, dg, None, None)


# ---- AdamW ----------------------------------------------------------------------------------

H = dict(lr=float(np.float32(1e-2)), beta1=float(np.float32(0.9)), beta2=float(np.float32(0.95)),
         eps=float(np.float32(1e-8)))
WD = float(np.float32(0.1))
SIZES = [1, 7, 8, 127, 128, 129, 2047, 2048, 2049, 5000, 0, 33, 3 * 2048 + 5]


def adamw_tensors(sizes, pdt, gdt, bits, master, seed=0):
    import mixture_experts_layer_router_amd as lm
    rng = np.random.default_rng(seed)
    p, g, mst = [], [], []
    for n in sizes:
        w = rng.standard_normal(n).astype(np.float32)
        p.append(put(w, pdt))
        mst.append(put(w) if master else None)
        g.append(put((rng.standard_normal(n) * np.exp(rng.uniform(-4, 0))).astype(np.float32), gdt))
    return lm.AdamW(p, g, masters=mst, state_bits=bits, weight_decay=WD, lr_scale=[1.0 if i % 2 else 0.5 for i in range(len(sizes))])


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("gdt", ["bf16", "f32"])
@pytest.mark.parametrize("pdt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_steps(bits, pdt, gdt, master):
    """Three steps over tensors of odd sizes, each against the oracle from the state before it.
    fp32 states: equal to the fp32 model of the oracle, every operation of which is rounded
    alike.  8 bits: the exponents equal the model's, the codes the model's for a quotient within
    two ulps.  The weight: the quotient and
    its factors take at most 12 roundings of the update and 3 of the weight, then the storage
    rounding."""
    import torch
    dt = dict(bf16=torch.bfloat16, f32=torch.float32)
    opt = adamw_tensors(SIZES, dt[pdt], dt[gdt], bits, master)
    gs = put(np.array([0.25], np.float32))
    for step in (1, 2, 3):
        say(f"adamw bits={bits} p={pdt} g={gdt} master={master} step {step}")
        before = [[None if t is None else t.clone() for t in x] for x in
                  (opt.params, opt.masters, opt.m, opt.v, opt.m_scales, opt.v_scales)]
        opt.step(step=step, seed=11, grad_scale=gs, **H)
        for i, n in enumerate(SIZES):
            if n == 0:
                continue
            w0 = to_np(before[1][i] if master else before[0][i]).astype(np.float64)
            g = to_np(opt.grads[i])
            if bits == 32:
                m0, v0 = to_np(before[2][i]), to_np(before[3][i])
            else:
                m0, r0 = (ot.e4m3_values(to_np(before[a][i])) * np.repeat(2.0 ** (to_np(before[a + 2][i]).astype(np.float64) - 127), 128)[:n]
                          for a in (2, 3))
                m0, v0 = m0.astype(np.float32), r0.astype(np.float32) ** 2
            m32, v32, r32 = ot.adamw_fp32(w0, g, m0, v0, step=step, wd=WD, grad_scale=0.25, **H)
            lr = H["lr"] * (1.0 if i % 2 else 0.5)
            w64, m64, v64 = ot.adamw(w0, g, m0.astype(np.float64), v0.astype(np.float64), lr, H["beta1"], H["beta2"], H["eps"],
                                     WD, step, 0.25)
            np.testing.assert_allclose(m32, m64, atol=4 * U * (np.abs(m0).max() + np.abs(g).max()))
            if bits == 32:
                np.testing.assert_array_equal(to_np(opt.m[i]), m32)
                np.testing.assert_array_equal(to_np(opt.v[i]), v32)
            else:
                u = ot.random_bits(11, step, i, np.arange(n))
                for val, b, low, q, k in ((m32, u & np.uint64(0xFFFF), False, opt.m[i], opt.m_scales[i]),
                                          (r32, u >> np.uint64(16), True, opt.v[i], opt.v_scales[i])):
                    # the value over 2^k is off by an ulp of the scale and a rounding at most
                    want = [ot.round_random(val, b, low, ulps) for ulps in (-2, -1, 0, 1, 2)]
                    np.testing.assert_array_equal(to_np(k), want[2][1] + 127)
                    assert np.any([to_np(q) == w[0] for w in want], axis=0).all()
                    # the neighbours differ for 2 in 2^20 of the random fractions
                    assert (to_np(q) != want[2][0]).sum() <= 2
            upd = np.abs(w64 - w0 * (1 - lr * WD))
            # cancellation in m: its error against its terms, over the same denominator
            terms = (np.abs(H["beta1"] * m0) + np.abs(0.1 * g * 0.25)) / (np.sqrt(v64 / (1 - H["beta2"] ** step)) + H["eps"])
            tol = 12 * U * upd + 4 * U * lr / (1 - H["beta1"] ** step) * terms + 3 * U * np.abs(w0) + 1e-37
            if master:
                got = to_np(opt.masters[i]).astype(np.float64)
                assert (np.abs(got - w64) <= tol).all()
                assert torch.equal(opt.params[i], opt.masters[i].to(dt[pdt]))
            else:
                got = to_np(opt.params[i]).astype(np.float64)
                assert (np.abs(got - w64) <= tol + (2.0 ** -8 if pdt == "bf16" else U) * (np.abs(w64) + tol)).all()


def test_adamw_many_tensors_and_order():
    """More tensors than one launch holds; each equals its step in a call with one tensor where
    no random bits are drawn, and the same call twice gives the same bits where they are."""
    import torch
    sizes = [5 + 37 * i for i in range(75)]
    f = torch.float32
    a = adamw_tensors(sizes, f, f, 32, False)
    b = adamw_tensors(sizes, f, f, 32, False)
    a.step(step=2, **H)
    import mixture_experts_layer_router_amd as lm
    for i in range(75):
        lm.AdamW([b.params[i]], [b.grads[i]], [b.m[i]], [b.v[i]], weight_decay=WD, lr_scale=1.0 if i % 2 else 0.5).step(step=2, **H)
        assert torch.equal(a.params[i], b.params[i]) and torch.equal(a.m[i], b.m[i]) and torch.equal(a.v[i], b.v[i])
    c, d = adamw_tensors(sizes, f, f, 8, False), adamw_tensors(sizes, f, f, 8, False)
    for o in (c, d):
        o.step(step=2, seed=5, **H)
    for x, y in ((c.params, d.params), (c.m, d.m), (c.v_scales, d.v_scales)):
        assert all(torch.equal(s, t) for s, t in zip(x, y))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_adamw_skips_a_step_that_is_not_finite(bits, value):
    import torch
    opt = adamw_tensors([300, 20], torch.bfloat16, torch.float32, bits, True)
    keep = [[t.clone() for t in x] for x in (opt.params, opt.masters, opt.m, opt.v)]
    opt.step(step=1, grad_scale=put(np.array([value], np.float32)), **H)
    for x, y in zip(keep, (opt.params, opt.masters, opt.m, opt.v)):
        assert all(torch.equal(s, t) for s, t in zip(x, y))


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_overflowing_square_moves_no_weight(bits):
    """A finite gradient whose square is infinite: v and its root are infinite, so by the formula
    that weight's update is 0 (m / infinity), in this step and in the next."""
    import torch
    import mixture_experts_layer_router_amd as lm
    n, at = 3000, 2222
    say(f"adamw {bits} bits, gradient 1e20")
    g = torch.full((n,), 0.5, device=device())
    g[at] = 1e20
    p = torch.ones(n, device=device())
    opt = lm.AdamW([p], [g], state_bits=bits)
    for step in (1, 2):
        opt.step(1e-2, step=step)
        w = to_np(p)
        assert w[at] == 1.0 and np.isfinite(w).all()
        assert (np.delete(w, np.s_[2176:2304]) < 1.0).all()
    if bits == 32:
        assert np.isinf(to_np(opt.v[0])[at]) and np.isfinite(np.delete(to_np(opt.v[0]), at)).all()


@pytest.mark.parametrize("big", [1e20, np.inf])
def test_adamw_8bit_overflow_stays_in_its_block(big):
    """v overflows in one block of 128: that block gets the largest exponent, the others are
    the bits of a step without it."""
    import torch
    import mixture_experts_layer_router_amd as lm
    say(f"adamw 8 bits, gradient {big}")
    rng = np.random.default_rng(21)
    n, at = 1000, 300  # block 2: 256..383
    g = rng.standard_normal(n).astype(np.float32)
    runs = []
    for value in (g[at], np.float32(big)):
        g[at] = value
        p = torch.ones(n, device=device())
        opt = lm.AdamW([p], [torch.tensor(g, device=device())], state_bits=8)
        for step in (1, 2):
            opt.step(1e-2, step=step, seed=3)
        runs.append([to_np(t) for t in (p, opt.m[0], opt.v[0], opt.m_scales[0], opt.v_scales[0])])
    out, blk = np.r_[0:256, 384:n], np.r_[0:2, 3:8]
    for a, b in zip(runs[0][:3], runs[1][:3]):
        np.testing.assert_array_equal(a[out], b[out])
    for a, b in zip(runs[0][3:], runs[1][3:]):
        np.testing.assert_array_equal(a[blk], b[blk])
    assert runs[1][4][2] == 247 and runs[1][2][at] == 126


def test_adamw_zero_gradients_and_betas():
    """Zero gradients on a new state: the weight only decays, the states stay zero (exponent
    byte 127); beta1 = beta2 = 0: m = g, v = g^2."""
    import torch
    opt = adamw_tensors([200], torch.float32, torch.float32, 8, False)
    opt.grads[0].zero_()
    w = to_np(opt.params[0]).astype(np.float64)
    opt.step(step=1, **H)
    assert not bool(opt.m[0].any()) and not bool(opt.v[0].any()) and bool((opt.m_scales[0] == 127).all())
    np.testing.assert_allclose(to_np(opt.params[0]), w * (1 - 0.5 * H["lr"] * WD), rtol=4 * U)
    opt = adamw_tensors([200], torch.float32, torch.float32, 32, False)
    g = to_np(opt.grads[0])
    opt.step(1e-3, beta1=0.0, beta2=0.0, eps=1e-8, step=1)
    np.testing.assert_array_equal(to_np(opt.m[0]), g)
    np.testing.assert_array_equal(to_np(opt.v[0]), g * g)


def test_adamw_leaves_neighbours_alone():
    """Bytes beside every buffer of an odd-sized tensor keep their values."""
    import torch
    import mixture_experts_layer_router_amd as lm
    n = 2048 + 131
    for bits in (32, 8):
        big = {}

        def part(name, dtype, size):
            full = torch.full((size + 64,), 77, device=device()).to(dtype)
            big[name] = (full, size)
            return full[:size]
        nb = -(-n // 128)
        p, g = part("p", torch.bfloat16, n), part("g", torch.bfloat16, n)
        sdt = torch.float32 if bits == 32 else torch.uint8
        m, v = part("m", sdt, n), part("v", sdt, n)
        ms, vs = part("ms", torch.uint8, nb), part("vs", torch.uint8, nb)
        for t, val in ((p, 1), (g, 0.5), (m, 0), (v, 0), (ms, 127), (vs, 127)):
            t.fill_(val)
        lm.AdamW([p], [g], [m], [v], [ms], [vs], state_bits=bits).step(step=1, **H)
        for name, (full, size) in big.items():
            assert bool((full[size:].float() == 77).all()), (bits, name)


# ---- together -------------------------------------------------------------------------------

def layer(seed=0, T=200, d=128, N=12, Z=4, K=4, I=96):
    import torch
    rng = np.random.default_rng(seed)
    E = N + Z
    b = torch.bfloat16
    return dict(x=put(rng.standard_normal((T, d)), b), wr=put((rng.standard_normal((E, d)) / np.sqrt(d)).astype(np.float32)),
                bias=put(np.zeros(E, np.float32)), wg=put(rng.standard_normal((N, I, d)) / np.sqrt(d), b),
                wu=put(rng.standard_normal((N, I, d)) / np.sqrt(d), b), wd=put(rng.standard_normal((N, d, I)) / np.sqrt(I), b),
                dy=put(rng.standard_normal((T, d)) / T, b), T=T, d=d, N=N, Z=Z, K=K, I=I)


def whole(c, ws, balance, z, mask=None):
    import mixture_experts_layer_router_amd as lm
    out = lm.forward(c["x"], c["wr"], c["bias"], c["wg"], c["wu"], c["wd"], c["K"], workspace=ws)
    return out, lm.layer_backward(c["x"], c["wr"], c["wg"], c["wu"], c["wd"], out, c["dy"], ws, balance, z, token_mask=mask)


def workspace(c):
    import mixture_experts_layer_router_amd as lm
    return lm.workspace_for(lm.make_shape(c["T"], c["d"], c["N"], c["Z"], c["K"], c["I"], lm.BF16), device())


@pytest.mark.parametrize("T", [1, 200, 700])
def test_layer_backward_against_the_oracle(T):
    """forward -> balance loss -> gates -> FFN -> router, one after another on the forward's
    workspace, against the oracle chain fed with the GPU's own picks, logits and rows."""
    import mixture_experts_layer_router_amd as lm
    say(f"layer backward T={T}")
    c = layer(T=T)
    ws = workspace(c)
    out, r = whole(c, ws, 0.05, 1e-3)
    f = lambda t: to_np(t).astype(np.float64)  # noqa: E731
    s = lm.forward_saved(c["x"], c["N"], c["Z"], c["K"], c["I"], ws)
    idx = to_np(out["topk_idx"])
    lg, x, wr = f(s["logits"]), f(c["x"]), f(c["wr"])
    # the saved logits are the router's: fp32 sums of d terms
    assert np.abs(lg - x @ wr.T).max() <= (c["d"] + 8) * U * (np.abs(x) @ np.abs(wr).T).max()
    bal = ot.balance_loss(lg, idx, float(np.float32(0.05)), float(np.float32(1e-3)))
    np.testing.assert_array_equal(to_np(r["load"]), bal["load"])
    np.testing.assert_array_equal(to_np(out["load"]), bal["load"][0])
    np.testing.assert_allclose(f(r["loss"]), bal["loss"], rtol=512 * U)
    slot = to_np(s["slot_row"])
    nnz = int(to_np(s["ffn_offsets"])[-1])
    rows = f(s["ffn_rows"][:max(nnz, 1)])
    dgate, mag = ot.gate_backward(x, rows, slot, f(c["dy"]))
    assert (np.abs(f(r["dgate"]) - dgate) <= (c["d"] / 64 + 18) * U * mag + 1e-37).all()
    from oracle import backward as ob
    experts = lambda e: (f(c["wg"][e]), f(c["wu"][e]), f(c["wd"][e]))  # noqa: E731
    dx, dw = ob.ffn_backward(x, f(c["dy"]), idx, f(out["topk_gate"]), experts, c["N"])
    ref = ot.router_backward(x, wr, lg, idx, dgate, aux=bal["dlogits"], add=dx)
    assert rel_l2(f(r["dx"]), ref["dx"]) <= 2e-2   # the FFN backward's own bound for bf16 layers
    assert rel_l2(f(r["dw_router"]), ref["dw_router"]) <= 1e-5
    for e in dw:
        for name, want in zip(("dw_gate", "dw_up", "dw_down"), dw[e]):
            assert rel_l2(f(r[name][e]), want) <= 2e-2


def test_training_run_and_bias_controller():
    """Steps of the whole layer with AdamW and the selection bias's controller: every state
    stays finite, the same run twice gives the same bits."""
    import torch
    import mixture_experts_layer_router_amd as lm
    final = []
    for _ in range(2):
        c = layer(seed=2)
        E = c["N"] + c["Z"]
        ws = workspace(c)
        names = ("wr", "wg", "wu", "wd")
        grads = [torch.zeros_like(c[n]) for n in names]
        masters = [None] + [c[n].float() for n in names[1:]]
        opt = lm.AdamW([c[n] for n in names], grads, masters=masters, state_bits=8, weight_decay=0.1)
        integral, prev = torch.zeros(E, device=device()), torch.zeros(E, device=device())
        target = torch.full((E,), 1.0 / E, device=device())
        for step in range(1, 5):
            out, r = whole(c, ws, 0.01, 1e-4)
            for dst, src in zip(grads, ("dw_router", "dw_gate", "dw_up", "dw_down")):
                dst.copy_(r[src])
            opt.step(1e-3, step=step, seed=9)
            lm.bias_update(r["load"][0].contiguous(), target, c["bias"], integral, prev, c["T"], c["K"], c["N"], 1e-3, 0.0, 0.0)
        state = [c[n] for n in names] + [c["bias"]] + opt.m + opt.v_scales
        assert all(bool(torch.isfinite(t.float()).all()) for t in state)
        final.append([t.clone() for t in state])
    assert all(torch.equal(a, b) for a, b in zip(*final))


def test_step_in_a_graph():
    """forward, losses, gradients and update captured into one graph with the step number and
    gradient scale on the device: every replay equals the eager step on the same state, with
    eager work in between."""
    import torch
    import mixture_experts_layer_router_amd as lm
    from mixture_experts_layer_router_amd import train as lt
    dev = device()
    say("whole step in a graph")

    def make():
        c = layer(seed=4)
        E = c["N"] + c["Z"]
        shape = lm.make_shape(c["T"], c["d"], c["N"], c["Z"], c["K"], c["I"], lm.BF16)
        e = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=dev)  # noqa: E731
        u8 = lambda n: torch.zeros(n, dtype=torch.uint8, device=dev)  # noqa: E731
        b = dict(ws=workspace(c), bws=u8(lt.lc_moe_balance_workspace_size(shape, 1)),
                 rws=u8(lt.lc_moe_router_backward_workspace_size(shape)), fws=u8(lm.lc_moe_backward_workspace_size(shape)),
                 y=torch.zeros_like(c["x"]), idx=e(c["T"], c["K"], dt=torch.int32), gate=e(c["T"], c["K"]),
                 load=e(E, dt=torch.int32), loss=e(2), bload=e(1, E, dt=torch.int32), prob=e(1, E), dl=e(c["T"], E),
                 dgate=e(c["T"], c["K"]), dx=torch.zeros_like(c["x"]))
        names = ("wr", "wg", "wu", "wd")
        grads = [torch.zeros_like(c[n]) for n in names]
        opt = lm.AdamW([c[n] for n in names], grads, state_bits=8, weight_decay=0.1)
        step, gs = torch.ones(1, dtype=torch.int32, device=dev), torch.full((1,), 0.5, device=dev)
        wts = lm._weights(c["wr"], c["bias"], c["wg"], c["wu"], c["wd"])
        saved = lm.forward_saved(c["x"], c["N"], c["Z"], c["K"], c["I"], b["ws"])

        def run():
            lm.lc_moe_forward(shape, c["x"], wts, b["y"], b["idx"], b["gate"], b["load"], b["ws"])
            lt.lc_moe_balance_loss(shape, lt.BalanceCoef(0.05, 1e-3), saved["logits"], b["idx"], None, 1, None, b["loss"],
                                   b["bload"], b["prob"], b["dl"], b["bws"])
            lt.lc_moe_gate_backward(shape, c["x"], saved["ffn_rows"], c["T"] * c["K"], saved["slot_row"], c["dy"], b["dgate"])
            lm.lc_moe_ffn_backward(shape, c["x"], wts, b["idx"], b["gate"], c["dy"], b["dx"], grads[1], grads[2], grads[3],
                                   b["fws"])
            lt.lc_moe_router_backward(shape, c["x"], c["wr"], saved["logits"], b["idx"], b["dgate"], b["dl"], b["dx"],
                                      b["dx"], grads[0], None, b["rws"])
            opt.step(1e-3, step_dev=step, seed=3, grad_scale=gs)
        state = [c[n] for n in names] + opt.m + opt.v + opt.m_scales + opt.v_scales + [b["dx"], b["loss"], b["dgate"]]
        return run, state, step, gs, c

    run_e, state_e, step_e, gs_e, ce = make()
    run_g, state_g, step_g, gs_g, cg = make()
    start = [t.clone() for t in state_g]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_g()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_g()
    for t, s in zip(state_g, start):
        t.copy_(s)
    for i in range(1, 5):
        for st, gs in ((step_e, gs_e), (step_g, gs_g)):
            st.fill_(i)
            gs.fill_(1.0 / i)
        ce["x"].mul_(-1.0)
        cg["x"].mul_(-1.0)
        g.replay()
        torch.cuda.synchronize()
        run_e()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(state_g, state_e)):
            assert torch.equal(a, b), (i, j)


def test_two_streams():
    """The operators on a stream of the caller's while another runs the same on other buffers."""
    import torch
    import mixture_experts_layer_router_amd as lm
    kw = dict(T=513, d=328, E=257, K=7, aux=True)
    a, b = router_inputs(kw, 1), router_inputs(kw, 2)
    call = lambda v: lm.router_backward(v[0], v[1], v[2], v[3], v[4], 200, dlogits_aux=v[5])  # noqa: E731
    want = [call(a), call(b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            ra = call(a)
        with torch.cuda.stream(s2):
            rb = call(b)
        torch.cuda.synchronize()
        for got, ref in zip((ra, rb), want):
            assert all(torch.equal(got[k], ref[k]) for k in ref)
