"""Tokens and places without a pick, forward and backward: what they hold is read nowhere, and they have no gradient.
Rows that must not be read hold NaN; results are compared with those of the same call on rows of zeros, bit for bit
(a term of 0 changes no sum)."""
import numpy as np
import pytest

from gpu_common import device, say, to_np
from test_gpu_block import f64, lm, put
from test_gpu_block_layer import layer, workspace

pytestmark = pytest.mark.gpu


def without(t, dead, value):
    import torch
    t = t.clone()
    t[torch.tensor(dead, device=device())] = value
    return t


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


DEAD = {"some": lambda T, rng: rng.random(T) < 0.3, "most": lambda T, rng: rng.random(T) < 0.97,
        "stages": lambda T, rng: np.arange(T) // 32 % 2 == 0, "all": lambda T, rng: np.ones(T, bool),
        "last": lambda T, rng: np.arange(T) >= T - 1, "none": lambda T, rng: np.zeros(T, bool)}
# few tokens, small tiles, wide tiles (bf16); one piece of the reduction and several
ROUTER = [(1, 264, 20), (40, 264, 77), (64, 1032, 96), (65, 264, 20), (777, 520, 96), (1300, 264, 16), (2100, 6144, 40)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E", ROUTER)
@pytest.mark.parametrize("dead", DEAD)
def test_router_backward_leaves_tokens_without_a_gradient_out(T, d, E, dt, dead):
    """Rows of zeros in dlogits_aux, no gradient from the gates: their tokens' rows of x are not read."""
    import torch
    say(f"router backward {T} {d} {E} {dt} {dead}")
    rng = np.random.default_rng(T + d)
    off = DEAD[dead](T, rng)
    x = put(rng.standard_normal((T, d)), torch.bfloat16 if dt == "bf16" else torch.float32)
    wr = put((rng.standard_normal((E, d)) / np.sqrt(d)).astype(np.float32))
    dl = rng.standard_normal((T, E)).astype(np.float32)
    dl[off] = 0.0
    if not off[0]:
        dl[0] = 0.0
        dl[0, E - 1] = 2.0 ** -100  # one term, small as it is, is a gradient
    dl = put(dl)
    for value in (float("nan"), float("inf")):
        bad, good = without(x, off, value), without(x, off, 0.0)
        got = lm().router_backward(bad, wr, None, None, None, E, dlogits_aux=dl)
        ref = lm().router_backward(good, wr, None, None, None, E, dlogits_aux=dl)
        assert torch.equal(got["dw_router"], ref["dw_router"]) and torch.equal(got["dx"], ref["dx"])
    want = f64(dl).T @ f64(good)
    mag = np.abs(f64(dl)).T @ np.abs(f64(good))
    assert (np.abs(f64(got["dw_router"]) - want) <= (T / 16 + 40) * 2.0 ** -24 * mag + 1e-37).all()
    if not off[0]:  # a token with a gradient counts, NaN too
        worse = without(bad, np.arange(T) == 0, float("nan"))
        assert bool(lm().router_backward(worse, wr, None, None, None, E, dlogits_aux=dl)["dw_router"][E - 1].isnan().all())


@pytest.mark.parametrize("T", [40, 300, 2100])
def test_padded_rows_of_nan_have_a_gradient(T):
    """A forward on padded rows of NaN, then its gradient with dy of NaN there: as on rows of zeros."""
    import torch
    say(f"gradient of a padded batch T={T}")
    c = layer(T=T) if T < 2000 else layer(T=T, d=6144, N=4, Z=2, K=2, I=64)
    keep = np.arange(T) % 3 != 1
    mask = put(keep.astype(np.uint8))
    gt = lm().Gating("sigmoid", 2, 1, 2, True, 2.0)
    runs = []
    for value in (float("nan"), 0.0):
        x, dy = without(c["x"], ~keep, value), without(c["dy"], ~keep, value)
        ws = workspace(c)
        out = lm().forward(x, c["wr"], c["bias"], c["wg"], c["wu"], c["wd"], c["K"], workspace=ws, gating=gt, token_mask=mask)
        for losses in ((0.0, 0.0), (0.1, 1e-3)):
            runs.append(dict(lm().layer_backward(x, c["wr"], c["wg"], c["wu"], c["wd"], out, dy, ws, *losses, token_mask=mask,
                                                 gating=gt), y=out["y"]))
    for a, b in zip(runs[:2], runs[2:]):
        for k, v in b.items():
            if v is not None:
                assert bool(torch.isfinite(a[k]).all()) and torch.equal(a[k], v), k
        assert not to_np(a["dx"])[~keep].any() and to_np(a["dx"])[keep].any() and to_np(a["dw_router"]).any()


@pytest.mark.parametrize("T", [40, 700, 2100])
def test_padded_batches_captured_and_replayed(T):
    """A graph of forward and gradient, replayed on batches that are padded in other places, with eager work and waiting
    between the replays: the eager calls' bits."""
    import torch
    say(f"padded batches captured T={T}")
    c = layer(T=T) if T < 2000 else layer(T=T, d=6144, N=4, Z=2, K=2, I=64)
    gt = lm().Gating("sigmoid", 2, 1, 2, True, 2.0)
    ws, mask = workspace(c), torch.ones(T, dtype=torch.uint8, device=device())
    x, dy = c["x"].clone(), c["dy"].clone()

    def step(ws):
        out = lm().forward(x, c["wr"], c["bias"], c["wg"], c["wu"], c["wd"], c["K"], workspace=ws, gating=gt, token_mask=mask)
        return dict(lm().layer_backward(x, c["wr"], c["wg"], c["wu"], c["wd"], out, dy, ws, 0.1, 1e-3, token_mask=mask,
                                        gating=gt), y=out["y"])

    batches = [np.arange(T) % 3 != 1, np.ones(T, bool), np.arange(T) < T // 2, np.arange(T) % 64 >= 32]

    def fill(keep):
        x.copy_(without(c["x"], ~keep, float("nan")))
        dy.copy_(without(c["dy"], ~keep, float("nan")))
        mask.copy_(put(keep.astype(np.uint8)))

    want = []
    for keep in batches:
        fill(keep)
        want.append({k: v.clone() for k, v in step(workspace(c)).items() if v is not None})
        assert all(bool(torch.isfinite(v).all()) for v in want[-1].values())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(ws)
    for turn in range(2 * len(batches)):
        i = turn % len(batches)
        fill(batches[i])
        g.replay()
        torch.cuda.synchronize()
        for k, v in want[i].items():
            assert torch.equal(out[k], v), (turn, k)
        step(workspace(c))  # eager work between
