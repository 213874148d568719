"""Experts switched off by NaN in a logit or a bias: never picked, nothing in a sum, as those of -infinity."""
import numpy as np
import pytest

from gpu_common import say, to_np
from test_gpu_block import check_select, gating_of, lm, put

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("groups", [1, 8])
@pytest.mark.parametrize("E", [16, 77, 96, 768, 4095])
def test_select_with_nan(score, renorm, groups, E):
    import torch
    if E % groups:
        groups = 7 if E == 77 else 9
    say(f"select with NaN {score} {renorm} {groups} {E}")
    rng = np.random.default_rng(E + groups)
    T, K = 40, 8
    lg = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    lg[1::2] = rng.integers(-1, 2, lg[1::2].shape)  # equal ones: decided in fp64
    lg[3] = 0.0
    off = rng.random((T, E)) < 0.4
    off[0], off[1], off[2, 3:] = True, False, True
    off[4:8, :E // groups] = True  # a group of them
    lg[off] = np.nan
    lg[5, off[5]] = np.where(np.arange(off[5].sum()) % 2, -np.inf, np.nan)
    b = (0.05 * rng.uniform(-1, 1, E)).astype(np.float32)
    bad = b.copy()
    bad[rng.random(E) < 0.2] = np.nan
    kw = dict(K=K, score=score, groups=groups, top_groups=max(groups // 2, 1), group_rank=2 if groups > 1 else 1,
              renorm=renorm, scale=1.5)
    for bias in (None, b, bad, np.full(E, np.nan, np.float32)):
        got = lm().select(put(lg), None if bias is None else put(bias), K, lm().Gating(**gating_of(kw)))
        with np.errstate(invalid="ignore"):
            idx, _ = check_select(kw, lg, bias, None, got)
        # as with -infinity in the place of NaN, bit for bit
        plain = lambda a: None if a is None else put(np.where(np.isnan(a), -np.inf, a).astype(np.float32))  # noqa: E731
        same = lm().select(plain(lg), plain(bias), K, lm().Gating(**gating_of(kw)))
        assert torch.equal(got[0], same[0]) and torch.equal(got[1], same[1])
        # the gradient: no term of an expert that is off
        dg = put(rng.standard_normal((T, K)).astype(np.float32))
        d = lm().select_backward(put(lg), got[0], dg, lm().Gating(**gating_of(kw)))
        ref = lm().select_backward(plain(lg), got[0], dg, lm().Gating(**gating_of(kw)))
        assert torch.equal(d, ref) and not to_np(d)[off].any()
