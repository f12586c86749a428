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
