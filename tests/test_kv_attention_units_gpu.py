"""Attention of batches of hundreds of short sequences: a block of the prompt
kernel walks many units, some of them without a second tile of rows."""
import numpy as np
import pytest
import torch

from kv_util import Batch, attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [4, 3])
def test_units_of_one_and_two_tiles(G, d):
    """Row groups of at most 128 rows (one tile) and of more in turn, 1 to 5
    steps each; the same bits every time."""
    g = np.random.default_rng(G + d)
    B = 400
    q = np.where(g.random(B) < 0.5, g.integers(17 // G + 1, 128 // G + 1, B), g.integers(128 // G + 1, 400 // G + 1, B))
    kv = q + np.where(g.random(B) < 0.5, 0, g.integers(0, 200, B))
    bt = Batch(q.tolist(), kv.tolist(), 2, d, 16, seed=d).to_gpu()
    a = attend(bt, 2 * G)
    for _ in range(5):
        b = attend(bt, 2 * G)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("d", [64, 128])
def test_factors_of_a_tile_that_comes_and_goes(d):
    """One key head and prompts of one step: every other unit lacks the second
    tile. Queries of very different sizes, so that another sequence's factors
    would show; the same bits every time."""
    g = np.random.default_rng(d)
    B, G = 600, 8
    q = g.integers(33, 49, B)
    bt = Batch(q.tolist(), q.tolist(), 1, d, 64, seed=d).to_gpu()
    x = g.standard_normal((bt.N, G, d)) * np.repeat(np.exp2(g.integers(-9, 3, B)), q)[:, None, None]
    a = attend(bt, G, q=x)
    for _ in range(5):
        b = attend(bt, G, q=x)
        assert all(torch.equal(y, z) for y, z in zip(a, b))
