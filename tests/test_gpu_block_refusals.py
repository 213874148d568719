"""What the block operators refuse of tensors on the GPU, each by its own message or status; nothing is written."""
import pytest

from gpu_common import device, say
from test_gpu_block import lm

pytestmark = pytest.mark.gpu


def test_a_linear_layer_over_its_input():
    import torch
    from mixture_experts_layer_router_amd import block as lb
    say("linear over its input")
    x = torch.ones((4, 16), dtype=torch.bfloat16, device=device())
    wq = lm().quantize_matrix(torch.full((16, 16), 2.0, dtype=torch.bfloat16, device=device()), transposed=True)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=device())
    with pytest.raises(ValueError, match="out overlaps"):
        lm().linear_fp8(x, wq, out=x)
    with pytest.raises(ValueError, match="out overlaps"):
        lm().linear_fp8_backward(x, x.clone(), wq, dx=x)
    for call in (lambda: lb.lc_moe_linear_fp8(4, 16, 16, x, wq.data, None, x, ws),
                 lambda: lb.lc_moe_linear_fp8_backward(4, 16, 16, x, x.clone(), wq.t, None, x, None, ws)):
        with pytest.raises(lm().LcMoeError) as e:
            call()
        assert e.value.status == 2  # LC_MOE_E_SHAPE
    torch.cuda.synchronize()
    assert bool((x == 1).all())


def test_workspaces_over_other_tensors():
    import torch
    say("workspaces over other tensors")
    b, one = torch.zeros(1 << 16, dtype=torch.bfloat16, device=device()), torch.ones(16, device=device())
    x = b[:64].view(4, 16)
    with pytest.raises(ValueError, match="workspace overlaps"):
        lm().block_norm_backward(x, one, x.clone(), workspace=b)
    for name in ("dz", "dh"):
        with pytest.raises(ValueError, match=f"{name}: shape"):
            lm().block_norm_backward(x, one, **{"dz": None, name: x[:3]})
    with pytest.raises(ValueError, match="rows or transposed"):
        lm().quantize_matrix(x, rows=False)


def test_the_gradient_of_a_weight_with_a_scale_for_each_row():
    import torch
    say("gradient of a weight with a scale for each row")
    w, x = torch.randn((16, 24), device=device()).bfloat16(), torch.randn((4, 24), device=device()).bfloat16()
    dy = torch.randn((4, 16), device=device()).bfloat16()
    m = lm().quantize_matrix(w, block_rows=1, transposed=True)
    assert m.block_rows == 1 and lm().quantize_matrix(w).block_rows == 128
    with pytest.raises(ValueError, match="block_rows 1"):
        lm().linear_fp8_backward(dy, x, m)
    assert "dx" not in lm().linear_fp8_backward(dy, x, m, need_dx=False)
