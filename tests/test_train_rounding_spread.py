"""How far the random rounding of the 8-bit states scatters them (the oracle's model, no GPU)."""
import numpy as np
import pytest

from oracle import train as ot


@pytest.mark.parametrize("b2", [0.999, 0.95])
def test_8bit_states_scatter_no_more_than_their_rounding(b2):
    """r = sqrt v over 200 steps against the same states in 64 bits: its mean ratio is 1 within 2%,
    and its spread is the roundings' own.  A value at distance a from its lower and z from its
    upper neighbour rounds with variance a z; a rounding's share of v decays by b2 a step, and a
    relative error of r is half of v's.  The sum of the shares over the steps is the variance of
    the ratio, to first order; 25% are left for the second order and for 1024 samples' own scatter
    (2% of the root a standard deviation)."""
    rng = np.random.default_rng(5)
    n = 1024
    scale = np.exp(rng.uniform(-3, 3, n))
    grid = np.unique(ot.e4m3_values(np.arange(127)))
    v64 = scale ** 2
    q, k = ot.round_random(np.sqrt(v64).astype(np.float32), np.full(n, 1 << 15), True)  # a start without chance:
    r8 = ot.e4m3_values(q) * 2.0 ** np.repeat(k, 128)[:n]
    v64 = r8 ** 2  # both from the rounded states
    var = np.zeros(n)  # of v
    for step in range(1, 201):
        g = 0.5 * scale * rng.standard_normal(n)
        v64 = b2 * v64 + (1 - b2) * g ** 2
        v8 = b2 * r8 ** 2 + (1 - b2) * g ** 2
        r = np.sqrt(v8).astype(np.float32)
        q, k = ot.round_random(r, ot.random_bits(1, step, 0, np.arange(n)) >> np.uint64(16), True)
        unit = 2.0 ** np.repeat(k, 128)[:n].astype(np.float64)
        y = r / unit
        low = grid[np.searchsorted(grid, y, side="right") - 1]
        high = grid[np.minimum(np.searchsorted(grid, y, side="right"), grid.size - 1)]
        var = b2 ** 2 * var + (2 * r) ** 2 * (y - low) * (high - y) * unit ** 2
        r8 = ot.e4m3_values(q) * unit
    ratio = r8 / np.sqrt(v64)
    own = np.sqrt(np.mean(var / (2 * v64) ** 2))
    print(b2, ratio.mean(), ratio.std(), own)
    assert abs(ratio.mean() - 1) <= 0.02
    assert ratio.std() <= 1.25 * own
