"""Digits of the training operators' results where common inputs do not show them: router
weights whose rows share a large part, that part cancelling in dx, and ones with rows of zeros;
the scales of 8-bit states; the step number on the device.

u = 2^-24 is half an fp32 step relative to the value; a bf16 result is rounded by 2^-8 at most.
"""
import numpy as np
import pytest

from gpu_common import device, rel_l2, say, to_np
from oracle import train as ot

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def put(a, dtype=None):
    import torch
    t = torch.tensor(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(device())


# ---- router backward: dx ----------------------------------------------------------------------

# few tokens, tiles of 128 x 128, wide tiles (384 of 128 x 256); fp32 beside them
FORMS = [dict(T=40, d=1032), dict(T=600, d=520), dict(T=2048, d=6144), dict(T=40, d=516, f32=True),
         dict(T=600, d=516, f32=True)]


def cancelling(rng, T):
    """[T,3] fp32 of 24 digits each, rows that sum to exactly 0: a, b and -(a + b)."""
    a = rng.integers(1 << 22, 1 << 23, (T, 2)).astype(np.float64)
    return (np.stack([a[:, 0], a[:, 1], -(a[:, 0] + a[:, 1])], axis=1) * 2.0 ** -23).astype(np.float32)


@pytest.mark.parametrize("kw", FORMS, ids=lambda k: f"T{k['T']}_d{k['d']}_{'f32' if k.get('f32') else 'bf16'}")
def test_router_dx_where_the_rows_share_a_large_part(kw):
    """W_r = 4096 c + noise, dlogits that sum to 0 over the experts: dx is made of the noise
    alone, and every digit that dlogits or W_r lose shows 4096 times as large.  No softmax is
    in the way (dlogits = dlogits_aux).  Two fp16 parts are off by 2^-23 of a value, the product
    of two low parts, left out, is 2^-22: 8 u of a product, and 3 E partial products are added;
    three bf16 parts leave out 4 u, with 6 E additions."""
    import torch
    import mixture_experts_layer_router_amd as lm
    T, d, E, half = kw["T"], kw["d"], 3, not kw.get("f32")
    say(f"router dx, rows with a shared part {kw}")
    rng = np.random.default_rng(T + d)
    aux = cancelling(rng, T)
    w = (4096.0 * rng.standard_normal(d) + rng.standard_normal((E, d))).astype(np.float32)
    x = torch.zeros(T, d, dtype=torch.bfloat16 if half else torch.float32, device=device())
    got = to_np(lm.router_backward(x, put(w), None, None, None, E, dlogits_aux=put(aux), need_dw=False)["dx"])
    w64, a64 = w.astype(np.float64), aux.astype(np.float64)
    want = a64 @ w64
    tol = (6 * E + 8 + 8) * U * (np.abs(a64) @ np.abs(w64))
    tol += 2.0 ** -8 * (np.abs(want) + tol) if half else U * np.abs(want)
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1, worst


@pytest.mark.parametrize("kw", [dict(T=40, d=1032), dict(T=600, d=520), dict(T=2048, d=6144)],
                         ids=lambda k: f"T{k['T']}_d{k['d']}")
def test_router_dx_of_a_bf16_layer_is_off_by_its_rounding_alone(kw):
    """Rows of W_r with a shared part ten times the rest, gradients of the gates through the
    softmax.  Rounding to nearest is uniform within half a step, so its root mean square is at
    most 2^-8 / sqrt(3) of the value; dlogits in fp32 are off by at most 336 u of terms of either
    sign (see test_gpu_train.py), which the shared part shows ten times as large: 2^-12 at most."""
    import torch
    import mixture_experts_layer_router_amd as lm
    T, d, E, K = kw["T"], kw["d"], 96, 6
    say(f"router dx, rms error {kw}")
    rng = np.random.default_rng(T)
    w = ((10.0 * rng.standard_normal(d) + rng.standard_normal((E, d))) / np.sqrt(d)).astype(np.float32)
    lg = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)
    dg = rng.standard_normal((T, K)).astype(np.float32)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=device())
    got = to_np(lm.router_backward(x, put(w), put(lg), put(idx), put(dg), E, need_dw=False)["dx"])
    want = ot.router_backward(np.zeros((T, d)), w.astype(np.float64), lg, idx, dg)["dx"]
    assert rel_l2(got, want) <= 2.0 ** -8 / np.sqrt(3) + 2.0 ** -12


def test_router_dx_with_a_row_of_zeros():
    """Many tokens: a row of zeros among small rows of W_r, an expert that is not in use yet, takes
    no digits from the others."""
    import torch
    import mixture_experts_layer_router_amd as lm
    T, d, E = 2048, 6144, 3
    say("router dx, a row of zeros")
    rng = np.random.default_rng(11)
    aux = cancelling(rng, T)
    w = np.ldexp(rng.standard_normal((E, d)), -40).astype(np.float32)
    w[1] = 0
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=device())
    got = to_np(lm.router_backward(x, put(w), None, None, None, E, dlogits_aux=put(aux), need_dw=False)["dx"])
    w64, a64 = w.astype(np.float64), aux.astype(np.float64)
    want = a64 @ w64
    tol = (6 * E + 8 + 8) * U * (np.abs(a64) @ np.abs(w64))
    tol += 2.0 ** -8 * (np.abs(want) + tol)
    assert (np.abs(got - want) / tol).max() <= 1


def test_router_dx_with_one_large_column():
    """Many tokens: one column of W_r 2^16 times the others, so that most of the second fp16 parts
    are below fp16's normal numbers: an operand is off by 2^-39 of its row's largest there, and
    no more."""
    import torch
    import mixture_experts_layer_router_amd as lm
    T, d, E = 2048, 6144, 3
    say("router dx, one large column")
    rng = np.random.default_rng(12)
    aux = cancelling(rng, T)
    w = (4096.0 * rng.standard_normal(d) + rng.standard_normal((E, d))).astype(np.float32)
    w[:, 1:] *= np.float32(2.0 ** -16)
    w[:, 0] = 4096.0 * 3.5
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=device())
    got = to_np(lm.router_backward(x, put(w), None, None, None, E, dlogits_aux=put(aux), need_dw=False)["dx"])
    w64, a64 = w.astype(np.float64), aux.astype(np.float64)
    want = a64 @ w64
    tol = (6 * E + 8 + 8) * U * (np.abs(a64) @ np.abs(w64)) + 2.0 ** -39 * (np.abs(a64) @ np.abs(w64).max(1))[:, None]
    tol += 2.0 ** -8 * (np.abs(want) + tol)
    assert (np.abs(got - want) / tol).max() <= 1


# ---- AdamW ------------------------------------------------------------------------------------

def test_8bit_codes_at_the_border_of_the_random_rounding():
    """The codes are those of the value over 2^k, exactly: with beta1 = beta2 = 0, m = g and
    sqrt(v) = |g|, so a gradient can put the quotient right at, and one fp32 step below, the
    point where the random bits carry into the code.  Blocks of 2^k from k = -40 to 40."""
    import torch
    import mixture_experts_layer_router_amd as lm
    say("adamw, codes at the border")
    ks = np.arange(-40, 41)
    n = ks.size * 128
    u = ot.random_bits(5, 1, 0, np.arange(n))
    rng = np.random.default_rng(1)
    for half, low in ((u & np.uint64(0xFFFF), False), (u >> np.uint64(16), True)):
        r = (half.astype(np.int64) << 4) + 8
        border = (1 << 20) - r - rng.integers(0, 2, n)  # the digits below the code's last place
        # a normal code in [2^-6, 256): exponent and three digits at random
        y = ((rng.integers(121, 135, n) << 23) | (rng.integers(0, 8, n) << 20) | border).astype(np.int32).view(np.float32)
        y[::128] = 448.0  # every block's largest: its exponent is k
        g = np.ldexp(y, np.repeat(ks, 128)).astype(np.float32)
        grad = put(g if low else np.where(np.arange(n) % 3 == 0, -g, g))
        opt = lm.AdamW([torch.zeros(n, device=device())], [grad], state_bits=8)
        opt.step(1e-3, beta1=0.0, beta2=0.0, eps=1e-8, step=1, seed=5)
        q, s = (opt.v[0], opt.v_scales[0]) if low else (opt.m[0], opt.m_scales[0])
        want, k = ot.round_random(to_np(grad), half, low)
        np.testing.assert_array_equal(k, ks)
        np.testing.assert_array_equal(to_np(s), ks + 127)
        np.testing.assert_array_equal(to_np(q), want)


def test_8bit_codes_are_those_of_the_state_in_64_bits():
    """2^26 elements against the formula in fp64, the random rounding among it: sqrt(v) to the bit
    (from v in fp32, 1 in 2^21 lies on the other side of its border: 32 here), m wherever its two
    terms have one sign (where they cancel, what fp32 loses is more than two of its steps)."""
    import torch
    import mixture_experts_layer_router_amd as lm
    n, dev = 1 << 26, device()
    say("adamw, codes in 64 bits")
    gen = torch.Generator(device=dev)
    gen.manual_seed(17)
    g = (1e-3 * torch.randn(n, generator=gen, device=dev)).to(torch.bfloat16)
    opt = lm.AdamW([torch.zeros(n, dtype=torch.bfloat16, device=dev)], [g], state_bits=8)
    b1, b2 = float(np.float32(0.9)), float(np.float32(0.95))
    opt.step(1e-3, beta1=b1, beta2=b2, eps=1e-8, step=1, seed=1)
    g.copy_(1e-3 * torch.randn(n, generator=gen, device=dev))
    half = lambda codes, scales: codes.view(torch.float8_e4m3fn).double() * torch.exp2(scales.double() - 127).repeat_interleave(128)  # noqa: E731
    m0, r0 = half(opt.m[0], opt.m_scales[0]), half(opt.v[0], opt.v_scales[0])
    opt.step(1e-3, beta1=b1, beta2=b2, eps=1e-8, step=2, seed=1)
    key = int(ot.mix(np.uint64((1 + 0x9E3779B9 * 2) & 0xFFFFFFFF)))
    key = int(ot.mix(np.uint64((key + 0x3C6EF373) & 0xFFFFFFFF)))
    x = (torch.arange(n, device=dev) + key) & 0xFFFFFFFF
    for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85)):
        x = ((x ^ (x >> shift)) * factor) & 0xFFFFFFFF
    x = x ^ (x >> 16)
    assert int(x[12345]) == int(ot.random_bits(1, 2, 0, np.array([12345]))[0])
    a, b = b1 * m0, (1 - b1) * g.double()
    m, r = a + b, (b2 * r0 ** 2 + (1 - b2) * g.double() ** 2).sqrt()
    for name, val, bits, codes, scales, ask in (("m", m, x & 0xFFFF, opt.m[0], opt.m_scales[0], a * b >= 0),
                                                ("r", r, x >> 16, opt.v[0], opt.v_scales[0], r > 0)):
        y = (val * torch.exp2(127 - scales.double()).repeat_interleave(128)).abs()
        step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
        q = torch.floor(y / step + (bits.double() + 0.5) / 65536) * step
        got = codes.view(torch.float8_e4m3fn).double().abs()
        if name == "r":
            q = q.clamp(min=2.0 ** -9)
        wrong = ask & (y >= 2.0 ** -6) & (got != q)
        assert int(wrong.sum()) == 0, (name, int(wrong.sum()))


HYPER = dict(beta1=0.9, beta2=0.95, eps=1e-8, seed=7)


def optimizer(bits, master=True):
    """Two tensors (one ends inside a strip and a block) whose states are not zero."""
    import torch
    import mixture_experts_layer_router_amd as lm
    rng = np.random.default_rng(bits)
    w = [rng.standard_normal(n).astype(np.float32) for n in (5000, 2048)]
    opt = lm.AdamW([put(a, torch.bfloat16) for a in w], [put(rng.standard_normal(a.size), torch.bfloat16) for a in w],
                   masters=[put(w[0]), None] if master else None, state_bits=bits, weight_decay=0.1)
    opt.step(1e-2, step=3, **HYPER)
    return opt


def state(opt):
    return [t for x in (opt.params, opt.masters, opt.m, opt.v, opt.m_scales, opt.v_scales) for t in x if t is not None]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("number", [1, 2, 7, 1000, 0, -3])
def test_a_step_number_on_the_device_is_the_one_of_the_host(bits, number):
    """Bias corrections and random bits alike; values below 1 are 1.  (Step 5 has another bias
    correction than each of these numbers, so one that is not read shows; the numbers next to 1000 have
    none, since 1 - 0.95^1000 is 1 in 64 bits.)"""
    import torch
    say(f"adamw {bits} bits, step {number} on the device")
    a, b, c = (optimizer(bits) for _ in range(3))
    a.step(1e-2, step=max(number, 1), **HYPER)
    b.step(1e-2, step_dev=put(np.array([number], np.int32)), **HYPER)
    c.step(1e-2, step=5, **HYPER)
    for s, t in zip(state(a), state(b)):
        assert torch.equal(s, t)
    assert not torch.equal(a.params[0], c.params[0])
    if bits == 8:
        assert not torch.equal(a.m[0], c.m[0]) and not torch.equal(a.v[0], c.v[0])


@pytest.mark.parametrize("bits", [8, 32])
def test_replays_of_a_captured_step_are_the_numbered_steps(bits):
    """A step captured with its number on the device, replayed with other work between, against
    eager steps that are given the number by the host."""
    import torch
    say(f"adamw {bits} bits, captured")
    a, b = optimizer(bits), optimizer(bits)
    number = torch.full((1,), 4, dtype=torch.int32, device=device())
    keep = [t.clone() for t in state(b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step(1e-2, step_dev=number, **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(1e-2, step_dev=number, **HYPER)
    for t, s in zip(state(b), keep):
        t.copy_(s)
    for i in range(4, 8):
        number.fill_(i)
        for o in (a, b):
            o.grads[0].mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        a.step(1e-2, step=i, **HYPER)
        torch.cuda.synchronize()
        for s, t in zip(state(a), state(b)):
            assert torch.equal(s, t), i


def test_8bit_step_of_several_large_tensors():
    """The first and last 1000 or so elements of tensors of many strips (of 2048) and odd ends, against
    the oracle, codes to the bit; a tensor of one element between them."""
    import torch
    import mixture_experts_layer_router_amd as lm
    sizes = [2048 * 9001 + 5, 1, 2048 * 4002 + 129, 2048 * 3403, 2048 * 2000 + 2047]
    say(f"adamw 8 bits, {sizes}")
    gen = torch.Generator(device=device())
    gen.manual_seed(3)
    g = [torch.randn(n, generator=gen, device=device()).to(torch.bfloat16) for n in sizes]
    opt = lm.AdamW([torch.ones(n, dtype=torch.bfloat16, device=device()) for n in sizes], g, state_bits=8)
    h = dict(lr=float(np.float32(1e-2)), beta1=float(np.float32(0.9)), beta2=float(np.float32(0.95)), eps=float(np.float32(1e-8)))
    opt.step(step=2, seed=6, **h)
    for i, n in enumerate(sizes):
        first = max(n - 1000, 0) // 128 * 128
        for a, z in ((0, min(n, 1024)), (first, n)):
            gr, zero = to_np(g[i][a:z]), np.zeros(z - a, np.float32)
            m32, _, r32 = ot.adamw_fp32(zero, gr, zero, zero, wd=0.0, step=2, **h)
            u = ot.random_bits(6, 2, i, np.arange(a, z))
            for val, b, low, q, s in ((m32, u & np.uint64(0xFFFF), False, opt.m[i], opt.m_scales[i]),
                                      (r32, u >> np.uint64(16), True, opt.v[i], opt.v_scales[i])):
                want, k = ot.round_random(val, b, low)
                np.testing.assert_array_equal(to_np(s[a // 128:-(-z // 128)]), k + 127)
                np.testing.assert_array_equal(to_np(q[a:z]), want)
            w = ot.adamw(np.ones(z - a), gr, zero.astype(np.float64), zero.astype(np.float64), h["lr"], h["beta1"], h["beta2"],
                         h["eps"], 0.0, 2)[0]
            assert (np.abs(to_np(opt.params[i][a:z]) - w) <= 2.0 ** -8 * np.abs(w) * (1 + 2.0 ** -7)).all()


# ---- one expert -------------------------------------------------------------------------------

@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("aux", [False, True])
def test_router_backward_of_one_expert(f32, aux):
    """E = 1: p = 1, so the gates' gradient does not reach the logits (p is off by 128 u, see
    test_gpu_train.py, and dlogits by 336 u of 2 |dp|); what the losses give passes through."""
    import torch
    import mixture_experts_layer_router_amd as lm
    T, d, K = 70, 40, 1
    say(f"router, one expert, f32={f32} aux={aux}")
    rng = np.random.default_rng(8)
    dt = torch.float32 if f32 else torch.bfloat16
    x, w = put(rng.standard_normal((T, d)), dt), put(rng.standard_normal((1, d)).astype(np.float32))
    lg, dg = put(rng.standard_normal((T, 1)).astype(np.float32)), put(rng.standard_normal((T, K)).astype(np.float32))
    au = put(rng.standard_normal((T, 1)).astype(np.float32)) if aux else None
    r = lm.router_backward(x, w, lg, put(np.zeros((T, K), np.int32)), dg, 1, dlogits_aux=au, need_dlogits=True)
    f = lambda t: to_np(t).astype(np.float64)  # noqa: E731
    dl = f(au) if aux else np.zeros((T, 1))
    err = 336 * U * 2 * np.abs(f(dg)) + U * np.abs(dl)
    assert (np.abs(f(r["dlogits"]) - dl) <= err).all()
    want = dl @ f(w)
    tol = err @ np.abs(f(w)) + 16 * U * np.abs(want)
    assert (np.abs(f(r["dx"]) - want) <= tol + (U if f32 else 2.0 ** -8) * (np.abs(want) + tol)).all()
    tol = err.T @ np.abs(f(x)) + (6 * T + 12) * U * (np.abs(dl).T @ np.abs(f(x)))
    assert (np.abs(f(r["dw_router"]) - dl.T @ f(x)) <= tol).all()
