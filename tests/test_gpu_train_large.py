"""The training operators where element offsets pass 2^32: the far end of each array against
plain torch arithmetic in fp64 on those rows alone."""
import numpy as np
import pytest
import torch

from gpu_common import device, rel_l2, say, to_np
from oracle import train as ot

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device=device())
    g.manual_seed(seed)
    return g


def test_balance_and_router_beyond_2_32_logits():
    """T E > 2^32: a pool of 4096 experts on 2^20 + 577 tokens.  The balance loss' gradient and
    the router's dx on the last tokens; dW against a sum over pieces of the tokens."""
    import mixture_experts_layer_router_amd as lm
    T, E, K, d = (1 << 20) + 577, 4096, 2, 64
    say(f"T={T} E={E}: {T * E} logits")
    g = gen(1)
    lg = torch.empty(T, E, device=device())
    for a in range(0, T, 1 << 17):
        lg[a:a + (1 << 17)].normal_(generator=g)
    idx = torch.randint(0, E, (T, K), generator=g, device=device(), dtype=torch.int32)
    r = lm.balance_loss(lg, idx, 2048, 0.5, 1e-3)
    load = torch.bincount(idx.reshape(-1).long(), minlength=E)
    assert torch.equal(r["load"][0].long(), load)
    u = float(np.float32(0.5)) * (E * load - K * T).double() / (K * T) / T
    rows = lg[-300:].double()
    p = torch.softmax(rows, 1)
    lse = torch.logsumexp(rows, 1, keepdim=True)
    want = p * (u - (p * u).sum(1, keepdim=True)) + 2 * float(np.float32(1e-3)) / T * lse * p
    # fp32 throughout: a few tens of roundings of terms of either sign (see test_gpu_train.py)
    assert rel_l2(to_np(r["dlogits"][-300:]), to_np(want)) <= 1e-5
    x = torch.randn(T, d, generator=g, device=device()).to(torch.bfloat16)
    w = torch.randn(E, d, generator=g, device=device()) / 8
    dg = torch.randn(T, K, generator=g, device=device())
    aux = r["dlogits"]
    o = lm.router_backward(x, w, lg, idx, dg, 2048, dlogits_aux=aux)
    dw = torch.zeros(E, d, dtype=torch.float64, device=device())
    for a in range(0, T, 1 << 15):
        p = torch.softmax(lg[a:a + (1 << 15)].double(), 1)
        dp = torch.zeros_like(p)
        dp.scatter_add_(1, idx[a:a + (1 << 15)].long(), dg[a:a + (1 << 15)].double())
        dl = p * (dp - (p * dp).sum(1, keepdim=True)) + aux[a:a + (1 << 15)].double()
        dw += dl.t().contiguous() @ x[a:a + (1 << 15)].double()
    dx = dl @ w.double()
    n = dx.shape[0]
    assert rel_l2(to_np(o["dx"][-n:]), to_np(dx)) <= 2.0 ** -8
    assert rel_l2(to_np(o["dw_router"]), to_np(dw)) <= 1e-5


def test_gate_beyond_2_32_row_elements():
    import mixture_experts_layer_router_amd as lm
    T, K, d = 60000, 12, 6144
    R = T * K
    say(f"gate: {R * d} row elements")
    g = gen(2)
    rows = torch.empty(R, d, dtype=torch.bfloat16, device=device())
    for a in range(0, R, 1 << 16):
        rows[a:a + (1 << 16)].normal_(generator=g)
    x = torch.randn(T, d, generator=g, device=device()).to(torch.bfloat16)
    dy = torch.randn(T, d, generator=g, device=device()).to(torch.bfloat16)
    slot = torch.arange(R, dtype=torch.int32, device=device()).view(T, K).flip(1).contiguous()
    got = lm.gate_backward(x, rows, slot, dy)
    for sl in (slice(0, 50), slice(T - 50, T)):
        want = (rows[slot[sl].long()].double() * dy[sl, None].double()).sum(-1)
        mag = (rows[slot[sl].long()].double() * dy[sl, None].double()).abs().sum(-1)
        assert bool(((got[sl].double() - want).abs() <= (d / 64 + 18) * 2.0 ** -24 * mag).all())


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_beyond_2_32_elements(bits):
    """The last 5000 elements of a tensor of 2^32 + 5000 against the oracle; the states of a
    stretch in the middle, whose gradients are zero, stay zero."""
    import mixture_experts_layer_router_amd as lm
    n, k = (1 << 32) + 5000, 5000
    say(f"adamw {bits} bits, {n} elements")
    p = torch.full((n,), 0.5, dtype=torch.bfloat16, device=device())
    grad = torch.zeros(n, dtype=torch.bfloat16, device=device())
    rng = np.random.default_rng(3)
    grad[-k:] = torch.tensor(rng.standard_normal(k), dtype=torch.bfloat16)
    opt = lm.AdamW([p], [grad], state_bits=bits)
    h = dict(lr=float(np.float32(1e-2)), beta1=float(np.float32(0.9)), beta2=float(np.float32(0.95)), eps=float(np.float32(1e-8)))
    opt.step(step=1, seed=4, **h)
    g = to_np(grad[-k:])
    z = np.zeros(k, np.float32)
    m32, v32, r32 = ot.adamw_fp32(z, g, z, z, wd=0.0, step=1, **h)
    if bits == 32:
        np.testing.assert_array_equal(to_np(opt.m[0][-k:]), m32)
        np.testing.assert_array_equal(to_np(opt.v[0][-k:]), v32)
    else:
        # whole blocks of 128: the tensor's last k elements begin inside one (2^32 is a multiple)
        u = ot.random_bits(4, 1, 0, np.arange(n - k, n))
        for val, b, low, q, s in ((m32, u & np.uint64(0xFFFF), False, opt.m[0], opt.m_scales[0]),
                                  (r32, u >> np.uint64(16), True, opt.v[0], opt.v_scales[0])):
            want = [ot.round_random(val, b, low, ulps) for ulps in (-2, -1, 0, 1, 2)]
            blocks = -(-k // 128)
            np.testing.assert_array_equal(to_np(s[-blocks:]), want[2][1] + 127)
            assert np.any([to_np(q[-k:]) == w[0] for w in want], axis=0).all()
            assert (to_np(q[-k:]) != want[2][0]).sum() <= 2
    mid = slice((1 << 31) - 4096, (1 << 31) + 4096)
    assert not bool(opt.m[0][mid].any()) and not bool(opt.v[0][mid].any())
    assert bool((p[mid] == 0.5).all())
    w64 = ot.adamw(np.full(k, 0.5), g, z.astype(np.float64), z.astype(np.float64), h["lr"], h["beta1"], h["beta2"], h["eps"], 0.0, 1)[0]
    assert (np.abs(to_np(p[-k:]) - w64) <= 2.0 ** -8 * np.abs(w64) * (1 + 2.0 ** -7)).all()
