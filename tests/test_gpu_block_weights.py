"""The forms that a weight is given in."""
import pytest

from gpu_common import device, say
from test_gpu_block import lm
from test_gpu_block_layer import layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["fp8", "fp8_act", "packed"])
def test_layer_on_picks_does_not_read_the_weights_that_another_form_replaces(form):
    """forward with a gating and forward_picks take tensors without storage for them, as forward does."""
    import torch
    say(f"weights in another form: {form}")
    c = layer(T=60, d=256, I=128)
    w = (c["wg"], c["wu"], c["wd"])
    if form == "packed":
        kw = dict(packed=lm().pack_weights(*w))
    else:
        kw = dict(fp8=lm().quantize_weights(*w), fp8_act=form == "fp8_act")
    gone = [t.to("meta") for t in w]
    gt = lm().Gating("sigmoid", renorm=True)
    for gating in (None, gt):
        want = lm().forward(c["x"], c["wr"], c["bias"], *w, c["K"], gating=gating, **kw)
        got = lm().forward(c["x"], c["wr"], c["bias"], *gone, c["K"], gating=gating, **kw)
        for k in want:
            assert torch.equal(got[k], want[k]), k
    got = lm().forward_picks(c["x"], want["topk_idx"], want["topk_gate"], *gone, c["Z"], **kw)
    assert torch.equal(got["y"], want["y"]) and torch.equal(got["load"], want["load"])
    with pytest.raises(ValueError, match="w_gate is on meta"):
        lm().forward_picks(c["x"], want["topk_idx"], want["topk_gate"], *gone, c["Z"])
