"""Gates and their gradient where terms cancel: one pick, equal and nearly equal gradients.

Tolerance.  With renorm the gradient of pick k is scale w_k sum_j w_j (dg_k - dg_j).  A difference has one
rounding, a share is off by at most 8 max|ls| + 32 of u = 2^-24 (test_gpu_block.py), two of them by twice that, a
chain of K <= 64 terms by K + 2, the products with scale, 1 - s and w_k by 8: below C = 16 max|ls| + 256 of u of the sum
of the terms' absolute values.  That sum is of differences, so it is as small as they are."""
import numpy as np
import pytest

from gpu_common import say, to_np
from oracle import block as ob
from test_gpu_block import U, f64, lm, ls_bound, put

pytestmark = pytest.mark.gpu


def case(T, E, K, seed=13):
    rng = np.random.default_rng(seed)
    lg = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    idx = np.argsort(rng.random((T, E)), 1)[:, :K].astype(np.int32)
    aux = (0.1 * rng.standard_normal((T, E))).astype(np.float32)
    return rng, lg, idx, aux


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E", [(1, 1), (33, 77), (65, 768), (9, 2049)])
def test_one_renormalised_gate_is_constant(score, T, E):
    """K = 1 with renorm: the gate is the scale, whatever the logits are; its gradient is 0, exactly."""
    say(f"one gate {score} {T} {E}")
    rng, lg, idx, aux = case(T, E, 1)
    dg = rng.standard_normal((T, 1)).astype(np.float32)
    g = lm().Gating(score, renorm=True, scale=2.5)
    got = lm().select_backward(put(lg), put(idx), put(dg), g)
    assert not to_np(got).any()
    got = lm().select_backward(put(lg), put(idx), put(dg), g, dlogits_aux=put(aux))
    np.testing.assert_array_equal(to_np(got), aux)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("K", [2, 5, 12, 64])
def test_equal_gradients_of_renormalised_gates_cancel(score, K):
    """The gates of a token sum to the scale: gradients that are all the same move nothing."""
    say(f"equal gradients {score} {K}")
    rng, lg, idx, aux = case(70, 96, K)
    idx[3, K // 2:] = -1  # fewer picks
    dg = np.repeat(rng.standard_normal((70, 1)), K, 1).astype(np.float32)
    got = lm().select_backward(put(lg), put(idx), put(dg), lm().Gating(score, renorm=True, scale=2.5), dlogits_aux=put(aux))
    np.testing.assert_array_equal(to_np(got), aux)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("K,apart", [(2, 2.0 ** -10), (3, 2.0 ** -20), (12, 2.0 ** -12), (64, 2.0 ** -8)])
def test_nearly_equal_gradients_of_renormalised_gates(score, K, apart):
    say(f"nearly equal gradients {score} {K} {apart}")
    T, E, scale = 200, 96, 2.5
    rng, lg, idx, _ = case(T, E, K)
    dg = (rng.standard_normal((T, 1)) * (1 + apart * rng.standard_normal((T, K)))).astype(np.float32)
    got = f64(lm().select_backward(put(lg), put(idx), put(dg), lm().Gating(score, renorm=True, scale=scale)))
    C = 16 * ls_bound(lg, idx, score) + 256
    rest = ob.scores(-np.asarray(lg, np.float64), "sigmoid")  # 1 - s
    for t in range(T):
        w = ob.pick_weights(ob.log_scores(lg[t, idx[t]], score))
        d = np.asarray(dg[t], np.float64)[:, None] - np.asarray(dg[t], np.float64)[None, :]
        f = scale * w * (rest[t, idx[t]] if score == "sigmoid" else 1.0)
        want, mag = f * (d @ w), f * (np.abs(d) @ w)
        over = np.abs(got[t, idx[t]] - want) - C * U * mag
        assert over.max() <= 1e-37, (t, over.max())
