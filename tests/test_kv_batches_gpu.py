"""The cache calls and attention on batches of many sequences (searches and
scans past their first 32 and 128 sequences), some of them empty, single
tokens beside prompts, and what a refused index leaves of its neighbours."""
import numpy as np
import pytest
import torch

import oracle.attention_oracle as AO
import rotation_post_quantization_b200 as rq
from kv_util import DEV, Batch, attend, bf16

pytestmark = pytest.mark.gpu


def ragged(B, seed, most=40, long=120):
    """New rows and lengths: empty sequences, single tokens, chunks."""
    g = np.random.default_rng(seed)
    kind = g.random(B)
    q = np.where(kind < 0.2, 0, np.where(kind < 0.6, 1, g.integers(2, most, B)))
    return q.tolist(), (q + np.where(g.random(B) < 0.4, 0, g.integers(0, long, B))).tolist()


def read_back(codes, scale, bt, b, lo, hi):
    """bf16(code * scale) of tokens lo .. hi - 1 of sequence b."""
    t = np.arange(lo, hi)
    page, slot = bt.table[b, t // bt.P], t % bt.P
    x = codes[page, :, slot].astype(np.float32) * scale[page].astype(np.float32)[:, :, None]
    return torch.from_numpy(x).to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [33, 129, 500])
def test_append_and_read(B, d):
    q, kv = ragged(B, B)
    bt = Batch(q, kv, 3, d, 16, seed=B, behind=4).to_gpu()
    g = np.random.default_rng(1)
    t, x = bf16(g.standard_normal((2, bt.N, 3, d)) * np.where(g.random((2, bt.N, 1, 1)) < 0.1, 3.0, 1.0))
    rq.respin_kv_append(bt.cache, t[0], t[1], bt.t_len, bt.t_table, cu=bt.t_cu)
    out = torch.full((2, bt.N, 3, d), 9.0, dtype=torch.bfloat16, device=DEV)
    rq.respin_kv_read(bt.cache, out[0], out[1], bt.t_len, bt.t_table, cu=bt.t_cu)
    assert rq.respin_device_status() == 0
    n = int(bt.cu[-1])
    out = out.cpu()
    for i, (codes, scale, tc, ts) in enumerate(((bt.kc, bt.ks, bt.cache.k, bt.cache.k_scale),
                                                (bt.vc, bt.vs, bt.cache.v, bt.cache.v_scale))):
        AO.append(codes, scale, x[i, :n], bt.cu, bt.kv_len, bt.table, 16)
        assert np.array_equal(tc.cpu().numpy(), codes)
        assert np.array_equal(ts.cpu().numpy().view(np.uint32), scale.view(np.uint32))
        want = torch.cat([read_back(codes, scale, bt, b, kv[b] - q[b], kv[b]) for b in range(B)])
        assert torch.equal(out[i, :n], want) and (out[i, n:] == 9).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [33, 129, 500])
def test_attention_mixed(B, d):
    """Single tokens and short chunks beside prompts: both kernels' sequences in one call."""
    q, kv = ragged(B, B + 1)
    bt = Batch(q, kv, 2, d, 16, seed=B, behind=3).to_gpu()
    attend(bt, 8)
    attend(bt, 8, window=20)


@pytest.mark.parametrize("use_cu", [False, True])
@pytest.mark.parametrize("B", [33, 129, 500])
def test_attention_single_tokens(B, use_cu):
    g = np.random.default_rng(B)
    kv = np.where(g.random(B) < 0.1, 0, g.integers(1, 400, B)).tolist()
    attend(Batch([1] * B, kv, 2, 128, 32, seed=B).to_gpu(), 8, use_cu=use_cu)


@pytest.mark.parametrize("where,i,bad,code", [
    ("t_table", (0, 2), 10 ** 6, 511), ("t_table", (0, 2), -1, 511), ("t_len", 0, 10 ** 6, 512), ("t_len", 0, -4, 512),
    ("t_len", 0, 7, 512), ("t_cu", 0, -2, 512)])
def test_refused_index_leaves_the_others_right(where, i, bad, code):
    """The other sequence's codes, scales and rows are the oracle's; the refused tokens' places keep what they held."""
    bt = Batch([20, 20], [40, 40], 2, 64, 16, seed=8).to_gpu()
    t, x = bf16(np.random.default_rng(3).standard_normal((2, 40, 2, 64)))
    getattr(bt, where)[i] = bad
    rq.respin_kv_append(bt.cache, t[0], t[1], bt.t_len, bt.t_table, cu=bt.t_cu)
    assert rq.respin_device_status() == code
    out = torch.full((2, 40, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    rq.respin_kv_read(bt.cache, out[0], out[1], bt.t_len, bt.t_table, cu=bt.t_cu)
    assert rq.respin_device_status() == code
    out = out.cpu()
    lost = [bt.table[0, 2]] if where == "t_table" else list(bt.table[0, :3])   # pages of refused tokens
    for j, (codes, scale, tc, ts) in enumerate(((bt.kc, bt.ks, bt.cache.k, bt.cache.k_scale),
                                                (bt.vc, bt.vs, bt.cache.v, bt.cache.v_scale))):
        was, was_s = codes.copy(), scale.copy()
        AO.append(codes, scale, x[j], bt.cu, bt.kv_len, bt.table, 16)
        codes[lost], scale[lost] = was[lost], was_s[lost]
        assert np.array_equal(tc.cpu().numpy(), codes) and np.array_equal(ts.cpu().numpy(), scale)
        assert torch.equal(out[j, 20:], read_back(codes, scale, bt, 1, 20, 40))
        first = 12 if where == "t_table" else 0   # tokens 20 .. 31 of the first sequence lie on page 1
        assert torch.equal(out[j, :first], read_back(codes, scale, bt, 0, 20, 20 + first))
        if where != "t_len" or bad != 7:
            assert (out[j, first:20] == 9).all()
