"""Attention over caches whose values are very small, very large, or zero over
whole pages, and over weights far apart: out and lse against the oracle."""
import numpy as np
import pytest

from kv_util import Batch, attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q,kv", [(1, 640), (60, 640), (1, 20000), (300, 3000)])
@pytest.mark.parametrize("power", [-126, -120, -100, 100])
def test_all_value_scales_small_or_large(power, q, kv):
    """1 / scale and the sum of the weights over it stay in binary32; lse does not depend on the values."""
    bt = Batch([q], [kv], 2, 128, 64, seed=kv)
    bt.vs[:] = np.float32(2.0 ** power) * (1 if power == -126 else 64 * bt.vs)
    attend(bt.to_gpu(), 4)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q,kv", [(1, 640), (60, 640), (1, 20000), (60, 3000)])
@pytest.mark.parametrize("power", [-110, -80, -40, 20])
def test_pages_of_zeros_beside_any_scale(power, q, kv, d):
    """A page of zeros has scale 0; its tokens still count in the sum."""
    bt = Batch([q], [kv], 2, d, 64, seed=power + 200)
    bt.vs[:] = np.float32(2.0 ** power) * 64 * bt.vs
    for p in (0, 3, 4, 7, kv // 64 - 1):
        z = bt.table[0, p]
        bt.vc[z], bt.vs[z] = 0, 0.0
    attend(bt.to_gpu(), 4)


@pytest.mark.parametrize("q", [1, 60])
def test_only_pages_of_zeros(q):
    bt = Batch([q, q], [700, 5000], 1, 128, 64, seed=3)
    bt.vc[:], bt.vs[:] = 0, 0.0
    attend(bt.to_gpu(), 4)


@pytest.mark.parametrize("q,kv", [(1, 640), (60, 640), (1, 20000), (60, 3000)])
def test_value_scales_far_apart(q, kv):
    """Within 2^62 of one another."""
    bt = Batch([q], [kv], 2, 128, 64, seed=kv + 1, v_spread=30.0)
    attend(bt.to_gpu(), 4)
