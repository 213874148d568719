"""Tokens and places without a pick, forward and backward: they have no gradient."""
import numpy as np
import pytest

from gpu_common import say, to_np
from test_gpu_block import f64, lm, put
from test_gpu_block_layer import layer, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [40, 300])
def test_places_without_a_pick_have_no_gate_gradient(T):
    """dgate of index -1 is 0: of a padded token, and of a token with fewer experts to pick than K.  The other
    places' are the product of dy with the pick's output."""
    say(f"gate gradient of padded tokens T={T}")
    c = layer(T=T)
    E = c["N"] + c["Z"]
    keep = np.arange(T) % 3 != 1
    bias = np.full(E, -np.inf, np.float32)
    bias[[1, c["N"] + 1, 5]] = 0.1  # three experts for four places, one of them without computation
    gt = lm().Gating("sigmoid", renorm=True)
    ws = workspace(c)
    out = lm().forward(c["x"], c["wr"], put(bias), c["wg"], c["wu"], c["wd"], c["K"], workspace=ws, gating=gt,
                       token_mask=put(keep.astype(np.uint8)))
    r = lm().layer_backward(c["x"], c["wr"], c["wg"], c["wu"], c["wd"], out, c["dy"], ws, gating=gt)
    idx, dgate = to_np(out["topk_idx"]), f64(r["dgate"])
    assert (idx[keep] == -1).sum() == keep.sum() and (idx[~keep] == -1).all()
    assert not dgate[idx == -1].any()
    saved = lm().forward_saved(c["x"], c["N"], c["Z"], c["K"], c["I"], ws)
    rows, slot, x, dy = f64(saved["ffn_rows"]), to_np(saved["slot_row"]), f64(c["x"]), f64(c["dy"])
    for t, k in zip(*np.nonzero(idx >= 0)):
        v = x[t] if idx[t, k] >= c["N"] else rows[slot[t, k]]
        assert abs(dgate[t, k] - v @ dy[t]) <= (c["d"] / 64 + 18) * 2.0 ** -24 * (np.abs(v) @ np.abs(dy[t]))


@pytest.mark.parametrize("T", [7, 250, 700])
@pytest.mark.parametrize("repeat", [False, True])
def test_permute_tells_places_without_a_pick_from_zero_experts(T, repeat):
    """slot_row: a row, -1 for a zero-computation pick, -2 for an index outside the pool."""
    say(f"permute T={T} repeat={repeat}")
    rng = np.random.default_rng(T)
    N, Z, K = 6, 3, 4
    idx = np.argsort(rng.random((T, N + Z)), 1)[:, :K].astype(np.int32)
    idx[rng.random((T, K)) < 0.3] = -1
    idx[0, 1:3] = N + Z, 2147483647
    if repeat:
        idx[T - 1] = 2
    got = lm().permute(put(rng.standard_normal((T, 8)).astype(np.float32)), put(idx), N, N + Z)
    slot = to_np(got["slot_row"])
    outside = (idx < 0) | (idx >= N + Z)
    assert (slot[outside] == -2).all() and (slot[(idx >= N) & ~outside] == -1).all()
    order = np.lexsort((np.arange(T * K), np.where((idx >= 0) & (idx < N), idx, N).reshape(-1)))
    ffn = ((idx >= 0) & (idx < N)).sum()
    want = np.empty(T * K, np.int64)
    want[order[:ffn]] = np.arange(ffn)
    np.testing.assert_array_equal(slot[(idx >= 0) & (idx < N)], want.reshape(T, K)[(idx >= 0) & (idx < N)])
