"""Small attention weights in numbers: what many tokens far below a dominant
one add to a row."""
import numpy as np
import pytest
import torch

import oracle.attention_oracle as AO
import rotation_post_quantization_b200 as rq
from kv_util import DEV, Batch, bf16, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("power", [-20, -24, -28])
@pytest.mark.parametrize("q", [1, 60])
def test_many_small_weights_beside_a_dominant_one(q, power, where):
    """One token of weight 1 whose value is 0, 40000 of weight 2^power whose
    values are not, in each of many equal sequences (of shared pages), so that
    a block walks whole contexts. Tolerance, half a step each: bf16 output 2^-8; a weight's
    fp16 2^-11 and its exponent 2^-16 of its part; fp16's floor, 2^-25 beside a
    largest weight of 2^6 at least, for every token: n 2^-31 of the largest."""
    n, d, P, B = 40000, 128, 64, 600 if q == 1 else 200
    bt = Batch([q], [n], 1, d, P, seed=2)
    bt.kc[:], bt.vc[:] = 0, 127
    bt.ks[:], bt.vs[:] = 1 / 127, 1 / 64
    t = min(n - q, int(where * n))   # every row sees it
    bt.kc[bt.table[0, t // P], 0, t % P, 0] = 127
    bt.vc[bt.table[0, t // P], 0, t % P] = 0
    bt.to_gpu()
    x = np.zeros((q, 2, d))
    x[..., 0] = -power * np.log(2)
    tq, q64 = bf16(x)
    out = torch.zeros(B * q, 2, d, dtype=torch.bfloat16, device=DEV)
    rq.respin_kv_attention(bt.cache, tq.repeat(B, 1, 1), bt.t_len.repeat(B), bt.t_table.repeat(B, 1), out,
                           workspace(bt.cache, 2, B * q, q), scale=1.0)
    assert rq.respin_device_status() == 0
    ref, _, spread, top = AO.attention(q64, bt.kc, bt.vc, bt.ks, bt.vs, bt.cu, bt.kv_len, bt.table, P, scale=1.0)
    top = np.full_like(top, 127 / 64)   # the dominant weight, 1 at most
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -16) * spread + n * 2.0 ** -31 * top[..., None]
    got = out.double().cpu().numpy().reshape(B, q, 2, d)
    assert (np.abs(got - ref) <= tol).all()
