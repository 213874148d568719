"""Kernels of the block operators that are chosen by size: every tile of the FP8 product, with its reduction in one
piece and in several, alone and two products in one launch, and every kernel of the norms' gradient.  Tolerances are
those of test_gpu_block.py; test_block_plan.py checks on the CPU that these sizes choose what they are listed for."""
import numpy as np
import pytest

from gpu_common import device, say
from test_gpu_block import A, B, EPS, HALF, U, check_norm_backward, f64, lm, norm_args, norm_inputs, put

pytestmark = pytest.mark.gpu

# (M, N, K): tile, several pieces.  Rows, columns and runs that end inside a tile, odd numbers of stages.
PRODUCTS = {(2100, 6152, 264): (0, False), (2040, 6152, 504): (0, False), (134, 8728, 14224): (0, True),
            (515, 3456, 19528): (0, True), (6200, 1320, 264): (1, False), (6144, 1320, 136): (1, False),
            (2048, 6144, 16384): (1, False), (8470, 904, 504): (1, False), (149, 5992, 13472): (1, True),
            (261, 3720, 13000): (1, True), (6345, 144, 10672): (1, True), (1000, 6144, 8200): (1, True),
            (1030, 4104, 1032): (2, False), (131, 12120, 200): (2, False), (66, 4248, 3016): (2, True),
            (1561, 72, 7560): (2, True), (777, 1032, 520): (3, False), (300, 776, 504): (3, False),
            (33, 2048, 3328): (3, True)}
# (T, k, n): tiles of dx and dw, whether one launch makes both
GRADIENTS = {(777, 1032, 520): (3, 3, True), (1030, 2056, 1032): (2, 2, True), (2100, 1032, 1032): (2, 3, False),
             (16384, 6144, 2048): (0, 1, False), (2056, 6200, 1544): (0, 1, False), (2056, 4104, 2120): (1, 1, False)}


def values(buf, R, C):
    """A block-FP8 matrix as it stands for, fp64 [R,C], by the layout of lc_moe_fp8_matrix_size."""
    import torch
    cp, rp = -(-C // 128) * 128, -(-R // 256) * 256
    codes = buf[:R * cp].view(torch.float8_e4m3fn).float().double()
    at = -(-R * cp // 256) * 256
    r = torch.arange(R, device=buf.device)
    k = buf[at:at + cp // 128 * rp].view(cp // 128, rp)[:, (r & ~127) + 4 * (r & 31) + (r >> 5 & 3)].t().long() - 127
    unit = (k + 1023 << 52).view(torch.float64)  # 2^k
    return (codes.view(R, cp // 128, 128) * unit[:, :, None]).view(R, cp)[:, :C]


def check(got, a, b, add=None):
    """The product of two matrices of fp64 values, as check_product of test_gpu_block.py."""
    c = a @ b.t().contiguous()
    err = 2.0 ** -11 * (c.abs() + ((a * a) @ (b * b).t().contiguous()).sqrt())
    if add is not None:
        c, err = c + add.double(), err + U * add.double().abs()
    over = (got.double() - c).abs() - err * (1 + HALF["bf16"]) - HALF["bf16"] * c.abs()
    assert float(over.max()) <= 1e-37, float(over.max())


def normal(seed, *size):
    import torch
    g = torch.Generator(device=device())
    g.manual_seed(seed)
    return torch.randn(size, generator=g, device=device())


def rows_of(seed, R, C):
    """bf16 rows of different sizes."""
    import torch
    return (normal(seed, R, C) * torch.exp2(2 * normal(seed + 1, R, 1))).to(torch.bfloat16)


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product_of_every_form(M, N, K):
    import torch
    say(f"product {M} {N} {K}: tile {PRODUCTS[M, N, K]}")
    a, b = rows_of(M, M, K), (normal(N, N, K) / K ** 0.5).to(torch.bfloat16)
    add = normal(K, M, N).to(torch.bfloat16)
    am, bm = lm().quantize_matrix(a, block_rows=1), lm().quantize_matrix(b)
    av, bv = values(am.data, M, K), values(bm.data, N, K)
    # a code is off by 2^-4 of the value, or by half the smallest step, 2^-10, of a unit of at most amax / 224
    amax = torch.nn.functional.pad(a.double().abs(), (0, -K % 128)).view(M, -1, 128).amax(2)
    near = a.double().abs() * 2.0 ** -4 + (amax * 2.0 ** -10 / 224).repeat_interleave(128, 1)[:, :K]
    assert bool(((av - a.double()).abs() <= near).all())
    got = lm().matmul_fp8(am, bm)
    check(got, av, bv)
    assert torch.equal(got, lm().matmul_fp8(am, bm))
    with_add = lm().matmul_fp8(am, bm, add=add)
    check(with_add, av, bv, add)
    over = add.clone()
    assert lm().matmul_fp8(am, bm, add=over, out=over) is over and torch.equal(over, with_add)


@pytest.mark.parametrize("M,N,K", [k for k, (form, _) in PRODUCTS.items() if form == 1])
def test_product_of_rows_with_scales_of_their_own(M, N, K):
    """192 columns of a tile start in the middle of a run of scales: every row of B with a scale of its own, so
    that a byte taken from another row shows."""
    import torch
    say(f"product {M} {N} {K}: a scale for each row")
    a, b = rows_of(1, M, K), rows_of(3, N, K)
    am, bm = lm().quantize_matrix(a, block_rows=1), lm().quantize_matrix(b, block_rows=1)
    check(lm().matmul_fp8(am, bm), values(am.data, M, K), values(bm.data, N, K))


@pytest.mark.parametrize("T,k,n", GRADIENTS)
def test_gradients_of_every_form(T, k, n):
    import torch
    say(f"gradients {T} {k} {n}: tiles {GRADIENTS[T, k, n]}")
    x, dy = rows_of(5, T, k), (1e-3 * rows_of(7, T, n).float()).to(torch.bfloat16)
    add = (1e-3 * normal(9, T, k)).to(torch.bfloat16)
    wq = lm().quantize_matrix((normal(11, n, k) / k ** 0.5).to(torch.bfloat16), transposed=True)
    dyq = lm().quantize_matrix(dy, block_rows=1, transposed=True)
    xq = lm().quantize_matrix(x, block_rows=1, rows=False, transposed=True)
    dyv, wv = values(dyq.data, T, n), values(wq.t, k, n)
    out = lm().linear_fp8_backward(dy, x, wq)
    check(out["dx"], dyv, wv)
    check(out["dw"], values(dyq.t, n, T), values(xq.t, k, T))
    more = lm().linear_fp8_backward(dy, x, wq, dx_add=add)
    check(more["dx"], dyv, wv, add)
    assert torch.equal(more["dw"], out["dw"])


# Widths on both sides of every border of the norms' gradient, rows enough for a workgroup to take several.
WIDTHS = [dict(T=600, d=6144, post=True, gate="channel"), dict(T=600, d=6152, post=True, gate="channel"),
          dict(T=530, d=6152, post=True, gate="token"), dict(T=700, d=7168, post=True, gate="token"),
          dict(T=520, d=7168), dict(T=601, d=8192, post=True, gate="channel"), dict(T=300, d=8192, gate="token"),
          dict(T=5, d=8192, post=True, gate="channel"), dict(T=560, d=8200, post=True, gate="token"),
          dict(T=1030, d=4100, post=True, gate="channel"), dict(T=800, d=1544, post=True, gate="channel")]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kw", WIDTHS, ids=lambda k: "_".join(f"{a}{v}" for a, v in k.items()))
def test_norm_gradient_of_every_width(kw, dt):
    import torch
    from mixture_experts_layer_router_amd import block as lb
    if dt == "bf16" and kw["d"] % 8:
        kw = dict(kw, d=kw["d"] + 4)
    say(f"norm backward {kw} {dt}")
    c = norm_inputs(kw, dt)
    T, d = c["h"][0].shape
    run = lambda: lm().block_norm_backward(c["h"][0], c["w_pre"][0], c["dz"][0], dh=c["dh"][0], residual_scale=A,  # noqa: E731
                                           block_scale=B, eps=EPS, **norm_args(c, 0))
    out = run()
    wgs = lb.lc_moe_block_norm_backward_workspace_size(T, d, lm().BF16 if dt == "bf16" else lm().F32) // (12 * d)
    check_norm_backward(c, dt, out, T, d, wgs)
    again = run()
    for k in out:
        assert torch.equal(out[k], again[k]), k
    # rows that a workgroup takes after another give what they give alone
    few = lambda t: None if t is None else t[-3:].clone()  # noqa: E731
    o = norm_args(c, 0)
    gate = o["gate"] if o["gate"] is None or o["gate"].dim() == 1 else few(o["gate"])
    last = lm().block_norm_backward(few(c["h"][0]), c["w_pre"][0], few(c["dz"][0]), dh=few(c["dh"][0]), y=few(o["y"]),
                                    w_post=o["w_post"], gate=gate, residual_scale=A, block_scale=B, eps=EPS)
    assert torch.equal(last["dx"], out["dx"][-3:]) and torch.equal(last["dy"], out["dy"][-3:])
