"""AdamW.step without the number of the step, or with one that its 32 bits cannot hold, is
refused: the first step's bias correction and random bits would be used in its place."""
import pytest

import mixture_experts_layer_router_amd as lm
from mixture_experts_layer_router_amd import train as lt


@pytest.fixture
def opt(monkeypatch):
    """An optimizer of no tensors whose call is recorded instead of made."""
    import torch
    o = lm.AdamW.__new__(lm.AdamW)
    o.device, o.state_bits, o._tensors, o.seen = torch.device("cpu"), 8, (), []
    monkeypatch.setattr(lt, "lc_moe_adamw", lambda tensors, count, hyper: o.seen.append((hyper.step, bool(hyper.step_dev))))
    return o


@pytest.mark.parametrize("kw", [dict(), dict(step=None), dict(step=0), dict(step=-1), dict(step=1 << 31),
                                dict(step=(1 << 32) + 1)])
def test_a_step_without_its_number_is_refused(opt, kw):
    with pytest.raises(ValueError, match="step"):
        opt.step(1e-3, **kw)
    assert not opt.seen


def test_a_step_with_its_number(opt):
    import torch
    opt.step(1e-3, step=1)
    opt.step(1e-3, step=(1 << 31) - 1)
    opt.step(1e-3, step_dev=torch.ones(1, dtype=torch.int32))
    assert [s for s, _ in opt.seen[:2]] == [1, (1 << 31) - 1] and [d for _, d in opt.seen] == [False, False, True]
