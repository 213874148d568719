"""Calls that the block operators' documentation allows beside those of the other tests."""
import numpy as np
import pytest

from gpu_common import device, say, to_np
from test_gpu_block import check_select, f64, lm, put
from test_gpu_block_forms import check, normal, rows_of, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 70, 600])
def test_route_select(T, dt):
    """The choice from the tokens is that of the logits left in the workspace, with padding and without a bias too; a
    padded row of NaN changes no other's."""
    import torch
    say(f"route_select T={T} {dt}")
    rng = np.random.default_rng(T)
    d, N, Z, K = 256, 20, 12, 5
    x = put(rng.standard_normal((T, d)), torch.bfloat16 if dt == "bf16" else torch.float32)
    w = put((rng.standard_normal((N + Z, d)) / 16).astype(np.float32))
    bias = put((0.05 * rng.uniform(-1, 1, N + Z)).astype(np.float32))
    keep = np.arange(T) % 4 != 3
    kw = dict(score="sigmoid", groups=4, top_groups=2, group_rank=2, renorm=True, scale=2.0)
    gt = lm().Gating(**kw)
    shape = lm().make_shape(T, d, N, Z, K, 8, x.dtype)
    for b in (bias, None):
        ws = lm().workspace_for(shape, device())
        idx, gate = lm().route_select(x, w, b, K, N, gt, workspace=ws)
        lg = lm().forward_saved(x, N, Z, K, 8, ws)["logits"].clone()
        assert float((lg.double() - x.double() @ w.double().t()).abs().max()) <= 1e-4
        check_select(dict(kw, K=K), to_np(lg), None if b is None else to_np(b), None, (idx, gate))
        bad = x.clone()
        bad[torch.tensor(~keep, device=device())] = float("nan")
        i2, g2 = lm().route_select(bad, w, b, K, N, gt, token_mask=put(keep.astype(np.uint8)))
        assert (to_np(i2)[~keep] == -1).all() and not to_np(g2)[~keep].any()
        k = torch.tensor(keep, device=device())
        assert torch.equal(i2[k], idx[k]) and torch.equal(g2[k], gate[k])


@pytest.mark.parametrize("T,k,n", [(1, 136, 264), (16, 1032, 72), (64, 520, 520), (777, 264, 520), (2100, 1032, 1032)])
def test_linear_with_a_scale_for_each_row_of_the_weight(T, k, n):
    """A weight quantised finer than in blocks of 128 rows is one too, in either way of multiplying."""
    say(f"linear with a scale for each row {T} {k} {n}")
    x, w = rows_of(3, T, k), rows_of(5, n, k)
    wq, xq = lm().quantize_matrix(w, block_rows=1), lm().quantize_matrix(x, block_rows=1)
    check(lm().linear_fp8(x, wq), values(xq.data, T, k), values(wq.data, n, k))


@pytest.mark.parametrize("R,C", [(129, 264), (1000, 136), (8, 2056)])
def test_a_transpose_as_an_operand(R, C):
    """The form along the columns is a matrix of its own: the product of a matrix's transpose with itself."""
    import torch
    say(f"transpose as an operand {R} {C}")
    x = rows_of(7, R, C)
    m = lm().quantize_matrix(x, block_rows=1, rows=False, transposed=True)
    a = lm().Fp8Matrix(C, R, m.t, None)
    got = lm().matmul_fp8(a, a)
    check(got, values(m.t, C, R), values(m.t, C, R))
    assert torch.equal(got, got.t())


def test_outputs_and_workspaces_of_the_caller():
    """The same results in buffers that a program keeps, used again and again."""
    import torch
    say("buffers of the caller")
    T, k, n = 300, 520, 264
    x, dy = rows_of(1, T, k), rows_of(3, T, n)
    w = lm().quantize_matrix((normal(5, n, k) / 20).to(torch.bfloat16), transposed=True)
    xq = lm().quantize_matrix(x, block_rows=1)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device=device())  # (NaN wherever it is read as a number)
    y, dx, z = (torch.empty((T, c), dtype=torch.bfloat16, device=device()) for c in (n, k, n))
    one = torch.ones(k, device=device())
    want = (lm().linear_fp8(x, w), lm().linear_fp8_backward(dy, x, w), lm().matmul_fp8(xq, w),
            lm().block_norm_backward(x, one, x, y=x, w_post=one))
    for _ in range(3):
        assert lm().linear_fp8(x, w, out=y, workspace=ws) is y and torch.equal(y, want[0])
        r = lm().linear_fp8_backward(dy, x, w, dx=dx, workspace=ws)
        assert r["dx"] is dx and torch.equal(dx, want[1]["dx"]) and torch.equal(r["dw"], want[1]["dw"])
        assert lm().matmul_fp8(xq, w, out=z, workspace=ws) is z and torch.equal(z, want[2])
        b = lm().block_norm_backward(x, one, x, y=x, w_post=one, workspace=ws)
        assert all(torch.equal(b[k], want[3][k]) for k in b)
