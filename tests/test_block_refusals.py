"""What the block operators' wrappers refuse, each by the message of the check that is meant (CPU): tensors off the GPU are
refused too, by another message and behind the others."""
import pytest
import torch

import mixture_experts_layer_router_amd as lm
from mixture_experts_layer_router_amd import block as lb

BF, F = torch.bfloat16, torch.float32
OFF_GPU = "run on the GPU"


def zeros(*size, dtype=BF):
    return torch.zeros(*size, dtype=dtype)


def turned(*size, dtype=BF):
    """Of this size, not contiguous."""
    return torch.zeros(*size[::-1], dtype=dtype).t()


def matrix(rows, cols, transposed=False):
    buf = lambda r, c: zeros(lb.lc_moe_fp8_matrix_size(r, c), dtype=torch.uint8)  # noqa: E731
    return lm.Fp8Matrix(rows, cols, buf(rows, cols), buf(cols, rows) if transposed else None)


def refused(what, call, error=ValueError):
    with pytest.raises(error, match=what):
        call()


def test_select():
    lg, b, mask, g = zeros(4, 16, dtype=F), zeros(16, dtype=F), zeros(4, dtype=torch.uint8), lm.Gating()
    run = lambda lg=lg, b=b, mask=mask: lm.select(lg, b, 2, g, token_mask=mask)  # noqa: E731
    refused(OFF_GPU, run)
    refused("bias: shape", lambda: run(b=b[:8]))
    refused("bias: torch", lambda: run(b=b.double()), TypeError)
    refused("logits must be contiguous", lambda: run(lg=turned(4, 16, dtype=F)))
    refused("token_mask: shape", lambda: run(mask=zeros(5, dtype=torch.uint8)))
    refused("token_mask: torch", lambda: run(mask=mask.bool()), TypeError)
    refused("bias is on meta", lambda: run(b=b.to("meta")))


def test_route_select():
    x, w, g = zeros(4, 16), zeros(12, 16, dtype=F), lm.Gating()
    ws = zeros(1 << 20, dtype=torch.uint8)
    run = lambda x=x, w=w, ws=None: lm.route_select(x, w, None, 2, 8, g, workspace=ws)  # noqa: E731
    refused(OFF_GPU, run)
    refused("w_router: shape", lambda: run(w=zeros(12, 8, dtype=F)))
    refused("x must be contiguous", lambda: run(x=turned(4, 16)))
    refused("workspace: a contiguous", lambda: run(ws=ws[::2]))
    both = zeros(1 << 12)
    refused("workspace overlaps", lambda: run(x=both[:64].view(4, 16), ws=both))


def test_select_backward():
    lg, idx, dg, g = zeros(4, 16, dtype=F), zeros(4, 2, dtype=torch.int32), zeros(4, 2, dtype=F), lm.Gating()
    run = lambda lg=lg, idx=idx, dg=dg, aux=None: lm.select_backward(lg, idx, dg, g, dlogits_aux=aux)  # noqa: E731
    refused(OFF_GPU, run)
    refused("topk_idx: torch", lambda: run(idx=idx.long()), TypeError)
    refused("topk_idx: shape", lambda: run(idx=idx[:3]))
    refused("dgate: shape", lambda: run(dg=zeros(4, 3, dtype=F)))
    refused("dlogits_aux: shape", lambda: run(aux=lg[:, :8]))
    refused("dlogits_aux must be contiguous", lambda: run(aux=turned(4, 16, dtype=F)))


def test_forward_picks():
    x, idx, gate = zeros(4, 16), zeros(4, 2, dtype=torch.int32), zeros(4, 2, dtype=F)
    wg, wd = zeros(3, 8, 16), zeros(3, 16, 8)

    def run(x=x, idx=idx, gate=gate, wg=wg, wu=wg, wd=wd):
        return lm.forward_picks(x, idx, gate, wg, wu, wd, 1)
    refused(OFF_GPU, run)
    refused("topk_gate: shape", lambda: run(gate=gate[:2]))
    refused("w_up: shape", lambda: run(wu=wg[:2]))
    refused("w_down: torch", lambda: run(wd=wd.float()), TypeError)
    refused("w_down must be contiguous", lambda: run(wd=zeros(3, 8, 16).transpose(1, 2)))


def test_forward_picks_with_weights_in_another_form():
    """The three matrices give the sizes then, and no more."""
    x, idx, gate = zeros(4, 16), zeros(4, 2, dtype=torch.int32), zeros(4, 2, dtype=F)
    wg, wd = zeros(3, 8, 16).to("meta"), zeros(3, 16, 8).to("meta")
    for form in ("fp8", "packed"):
        run = lambda wu=wg: lm.forward_picks(x, idx, gate, wg, wu, wd, 1, **{form: zeros(64, dtype=torch.uint8)})  # noqa: E731
        refused(OFF_GPU, run)
        refused("w_up: shape", lambda: run(wu=wd))
    refused("w_gate is on meta", lambda: lm.forward_picks(x, idx, gate, wg, wg, wd, 1))


def test_block_norm():
    x, w = zeros(4, 16), zeros(16, dtype=F)
    run = lambda x=x, w=w, **kw: lm.block_norm(x, w, **kw)  # noqa: E731
    refused(OFF_GPU, run)
    refused("y: shape", lambda: run(y=x[:2]))
    refused("y must be contiguous", lambda: run(y=turned(4, 16)))
    refused("gate: shape", lambda: run(y=x, gate=zeros(4, 2, dtype=F)))
    refused("gate: shape", lambda: run(y=x, gate=zeros(4, dtype=F)))
    refused("w_pre: shape", lambda: run(w=w[:8]))
    refused("w_post: torch", lambda: run(y=x, w_post=w.to(BF)), TypeError)
    refused("need y", lambda: run(gate=w), TypeError)
    refused(OFF_GPU, lambda: lm.block_norm_backward(x, w, x))


def test_products():
    x, m = zeros(4, 16), matrix(8, 16)
    run = lambda x=x, m=m, **kw: lm.linear_fp8(x, m, **kw)  # noqa: E731
    refused(OFF_GPU, run)
    refused("x: shape", lambda: run(x=zeros(4, 8)))
    refused("x must be contiguous", lambda: run(x=turned(4, 16)))
    refused("add: shape", lambda: run(add=zeros(4, 16)))
    refused("w: shape", lambda: run(m=lm.Fp8Matrix(8, 16, m.data[:-1], None)))
    both = zeros(80)
    add, out = both[:32].view(4, 8), both[8:40].view(4, 8)  # part of one over part of the other
    refused("out overlaps", lambda: run(add=add, out=out))
    refused("out overlaps", lambda: run(x=both[:64].view(4, 16), out=out))
    refused("out overlaps", lambda: lm.linear_fp8(x, matrix(16, 16), out=x))  # over the tokens, whole
    refused(OFF_GPU, lambda: run(add=out, out=out))  # the addend itself
    a = matrix(4, 16)
    refused(OFF_GPU, lambda: lm.matmul_fp8(a, m))
    refused("columns", lambda: lm.matmul_fp8(matrix(4, 24), m))
    refused("out overlaps", lambda: lm.matmul_fp8(a, m, add=add, out=out))
    refused("out overlaps", lambda: lm.matmul_fp8(a, m, out=a.data[:64].view(BF).view(4, 8)))
    refused("lacks the form", lambda: lm.linear_fp8_backward(zeros(4, 8), x, m), TypeError)
    t = matrix(8, 16, transposed=True)
    back = lambda dy=zeros(4, 8), **kw: lm.linear_fp8_backward(dy, x, t, **kw)  # noqa: E731
    refused(OFF_GPU, back)
    refused("dy: shape", lambda: back(dy=zeros(3, 8)))
    wide = zeros(80)
    refused("out overlaps", lambda: back(dx_add=wide[:64].view(4, 16), dx=wide[8:72].view(4, 16)))
    refused("out overlaps", lambda: back(dy=wide[:32].view(4, 8), dx=wide[:64].view(4, 16)))
    refused("x: torch", lambda: lm.quantize_matrix(zeros(4, 16, dtype=F)), TypeError)
    refused("x must be contiguous", lambda: lm.quantize_matrix(turned(4, 16)))


def test_the_gradient_of_a_weight_with_a_scale_for_each_row():
    """Its transpose has scales for its columns, so it holds other values than the weight that was multiplied by."""
    x, dy, w = zeros(4, 16), zeros(4, 8), matrix(8, 16, transposed=True)
    rows = lm.Fp8Matrix(8, 16, w.data, w.t, block_rows=1)
    refused("block_rows 1", lambda: lm.linear_fp8_backward(dy, x, rows))
    refused(OFF_GPU, lambda: lm.linear_fp8_backward(dy, x, rows, need_dx=False))  # dw does not read it
    refused(OFF_GPU, lambda: lm.linear_fp8_backward(dy, x, w))
    refused(OFF_GPU, lambda: lm.linear_fp8(x, rows))
