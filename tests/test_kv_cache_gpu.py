"""The 8-bit paged cache: written codes and scales equal the oracle's bit for
bit, reading back gives bf16(code * scale), and the head norms and rotation
agree with float64."""
import numpy as np
import pytest
import torch

import oracle.attention_oracle as AO
import rotation_post_quantization_b200 as rq
from kv_util import DEV, Batch, attend, bf16

pytestmark = pytest.mark.gpu


def new_values(bt, seed, gain=1.0):
    g = np.random.default_rng(seed)
    x = g.standard_normal((2, bt.N, bt.H, bt.d)) * gain * np.where(g.random((2, bt.N, 1, 1)) < 0.1, 3.0, 1.0)
    return bf16(x)


def check_append(bt, t, x, use_cu=True, ld=None):
    n = int(bt.cu[-1])
    bt.to_gpu()
    rq.respin_kv_append(bt.cache, t[0], t[1], bt.t_len, bt.t_table, cu=bt.t_cu if use_cu else None)
    torch.cuda.synchronize()
    assert rq.respin_device_status() == 0
    for codes, scale, y, tc, ts in ((bt.kc, bt.ks, x[0], bt.cache.k, bt.cache.k_scale),
                                    (bt.vc, bt.vs, x[1], bt.cache.v, bt.cache.v_scale)):
        AO.append(codes, scale, y[:n], bt.cu, bt.kv_len, bt.table, bt.P)
        assert np.array_equal(ts.cpu().numpy().view(np.uint32), scale.view(np.uint32))
        assert np.array_equal(tc.cpu().numpy(), codes)   # untouched slots and pages too


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens", [([1] * 6, [1, 2, 16, 17, 128, 301]), ([5, 1, 130, 40], [5, 65, 400, 41]),
                                            ([300], [300]), ([0, 7, 0, 33, 0], [9, 7, 0, 70, 128])])
def test_append(q_lens, kv_lens, d, P):
    bt = Batch(q_lens, kv_lens, 3, d, P, seed=P, behind=2)
    t, x = new_values(bt, 1)
    check_append(bt, t, x)


@pytest.mark.parametrize("gain", [0.0, 1e-39, 1e-37, 1e-30, 1e30, 3e38])
def test_append_sizes(gain):
    """Zeros and values whose scale leaves binary32's normal numbers, and the largest bf16."""
    bt = Batch([1, 20], [9, 20], 2, 64, 16, seed=3)
    bt.ks[:] *= 1e-30
    g = np.random.default_rng(5)
    t, x = bf16(np.clip(g.standard_normal((2, bt.N, 2, 64)), -1, 1) * gain)
    check_append(bt, t, x)


def test_append_not_finite():
    bt = Batch([1, 20, 1], [9, 20, 1], 2, 64, 16, seed=4)
    x = np.random.default_rng(6).standard_normal((2, bt.N, 2, 64))
    x[0, 0, 0, 3], x[1, 2, 1, 5], x[0, 5, 0, 0] = np.nan, np.inf, -np.inf
    x[0, -1], x[1, -1] = np.nan, np.inf   # a page of nothing else
    t, y = bf16(x)
    check_append(bt, t, y)
    assert np.isfinite(bt.ks).all() and np.isfinite(bt.vs).all()


def test_append_uniform_and_strided():
    bt = Batch([3, 3, 3], [3, 20, 64], 2, 128, 16, seed=5)
    wide = torch.randn(9, 10, 128, device=DEV).bfloat16()
    t = (wide[:, 4:6], wide[:, 7:9])
    check_append(bt, t, [y.double().cpu().numpy() for y in t], use_cu=False)


def test_append_again_changes_nothing_and_token_by_token_grows():
    bt = Batch([40], [40], 2, 128, 64, seed=6)
    t, x = new_values(bt, 2)
    check_append(bt, t, x)
    before = [y.clone() for y in bt.cache]
    rq.respin_kv_append(bt.cache, t[0], t[1], bt.t_len, bt.t_table)
    assert all(torch.equal(a, b) for a, b in zip(before, bt.cache))
    one = Batch([1], [1], 2, 128, 64, seed=6)
    one.table = bt.table
    for n in range(1, 41):   # the same tokens one at a time: codes move with the scale
        one.kv_len = np.array([n], np.int32)
        one.kv_lens = [n]
        check_append(one, t[:, n - 1:n], x[:, n - 1:n])
    assert np.array_equal(one.ks.view(np.uint32)[bt.table[0, 0]], bt.ks.view(np.uint32)[bt.table[0, 0]])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("lens", [[1], [5, 0, 333, 16, 17], [100, 31]])
def test_read(lens, P, d):
    bt = Batch(lens, lens, 3, d, P, seed=7, behind=3).to_gpu()
    k = torch.full((bt.N, 3, d), 9.0, dtype=torch.bfloat16, device=DEV)
    wide = torch.full((bt.N, 5, d), 9.0, dtype=torch.bfloat16, device=DEV)
    rq.respin_kv_read(bt.cache, k, wide[:, 1:4], bt.t_len, bt.t_table, cu=bt.t_cu)
    assert rq.respin_device_status() == 0
    n = sum(lens)
    for got, codes, scale in ((k, bt.kc, bt.ks), (wide[:, 1:4], bt.vc, bt.vs)):
        want = np.concatenate([(c * s[:, :, None]) for b, m in enumerate(lens) for c, s in [_tokens(bt, codes, scale, b, m)]])
        want = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(got[:n].cpu(), want) and (got[n:] == 9).all()
    assert (wide[:, 0] == 9).all() and (wide[:, 4] == 9).all()


def _tokens(bt, codes, scale, b, m):
    page, slot = bt.table[b, np.arange(m) // bt.P], np.arange(m) % bt.P
    return codes[page, :, slot].astype(np.float32), scale[page].astype(np.float32)


def test_refused_indexes_are_recorded():
    bt = Batch([20, 20], [40, 40], 2, 64, 16, seed=8)
    t, x = new_values(bt, 3)
    for where, i, bad, code in (("t_table", (0, 2), 10 ** 6, 511), ("t_table", (0, 2), -1, 511), ("t_len", 0, 10 ** 6, 512),
                                ("t_len", 0, -4, 512), ("t_len", 0, 7, 512), ("t_cu", 0, -2, 512), ("t_cu", 1, 41, 512)):
        bt.to_gpu()
        getattr(bt, where)[i] = bad
        rq.respin_kv_append(bt.cache, t[0], t[1], bt.t_len, bt.t_table, cu=bt.t_cu)
        assert rq.respin_device_status() == code, (where, bad)
        other = bt.table[1, 0]
        assert np.array_equal(bt.cache.k[other].cpu().numpy(), bt.kc[other])   # a page of nobody's new tokens
        out = torch.full((40, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV)
        rq.respin_kv_read(bt.cache, out, out.clone(), bt.t_len, bt.t_table, cu=bt.t_cu)
        assert rq.respin_device_status() == code, (where, bad)


@pytest.mark.parametrize("N", [1, 3, 700])
@pytest.mark.parametrize("Hq,Hk,d,rot,qn,kn,inter", [
    (32, 8, 128, 128, True, True, False), (4, 4, 64, 64, False, False, False), (7, 1, 64, 32, True, False, True),
    (5, 3, 128, 64, False, True, False), (2, 1, 128, 128, False, False, True), (3, 2, 64, 16, True, True, False),
    (3, 0, 128, 128, True, False, False), (2, 2, 128, 0, True, True, False)])
def test_norm_rope(N, Hq, Hk, d, rot, qn, kn, inter):
    """Tolerance: the bf16 rounding (2^-8 of the value) and fp32's: sine and
    cosine of a reduced angle (2^-22 of the pair's length), the norm (sum,
    root, two products: 2^-20)."""
    g = np.random.default_rng(N + Hq)
    wide = torch.from_numpy(g.standard_normal((N, Hq + Hk + 1, d)).astype(np.float32)).bfloat16().to(DEV)
    q, k = wide[:, :Hq], wide[:, Hq:Hq + Hk]
    pos = g.integers(0, 1 << 20, N).astype(np.int32)
    pos[0] = -77
    freq = (10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
    w = [bf16(1 + 0.3 * g.standard_normal(d)) for _ in range(2)]
    qo, ko = torch.empty(N, Hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(N, Hk, d, dtype=torch.bfloat16, device=DEV)
    args = dict(q_weight=w[0][0] if qn else None, k_weight=w[1][0] if kn else None, eps=1e-5, interleaved=inter)
    x64 = wide.double().cpu().numpy()
    tp, tf = torch.from_numpy(pos).to(DEV), torch.from_numpy(freq).to(DEV)
    rq.respin_qk_norm_rope(q, k, tp, tf, qo, ko, **args)
    torch.cuda.synchronize()
    for got, x, on, ww in ((qo, x64[:, :Hq], qn, w[0][1]), (ko, x64[:, Hq:Hq + Hk], kn, w[1][1])):
        ref, amp = AO.norm_rope(x, ww if on else None, 1e-5, pos, freq, inter)
        assert (np.abs(got.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * amp).all()
    rest = wide[:, Hq + Hk:].clone()
    rq.respin_qk_norm_rope(q, k, tp, tf, q, k, **args)   # in place
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(wide[:, Hq + Hk:], rest)


@pytest.mark.parametrize("gain", [0.0, 1e-30, 1e25, 3e38])
def test_norm_sizes(gain):
    """Squares below and above binary32."""
    g = np.random.default_rng(1)
    t, x = bf16(g.uniform(0.5, 1.0, (3, 2, 64)) * gain)
    w, w64 = bf16(np.ones(64))
    out, ko = torch.empty_like(t), torch.empty_like(t)
    z = torch.zeros(3, dtype=torch.int32, device=DEV)
    rq.respin_qk_norm_rope(t, t, z, torch.zeros(0, device=DEV), out, ko, q_weight=w, k_weight=w, eps=1e-6)
    ref, _ = AO.norm_rope(x, w64, 1e-6, np.zeros(3), np.zeros(0), False)
    assert (np.abs(out.double().cpu().numpy() - ref) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(ref)).all()
    assert torch.equal(out, ko)


def test_steps_of_a_sequence_together():
    """Prefill, then decode steps: rotation, append and attention run on one
    stream as a layer runs them, each step checked against the oracle on the
    cache as it stands."""
    H, G, d, P = 2, 4, 128, 16
    g = np.random.default_rng(2)
    lens = [37, 64, 5]
    bt = Batch(lens, [n + 8 for n in lens], H, d, P, seed=1).to_gpu()   # pages for 8 more tokens
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, d, 2) / d)).astype(np.float32)).to(DEV)
    w, w64 = bf16(1 + 0.2 * g.standard_normal(d))
    for step in range(4):
        bt.q_lens = lens if step == 0 else [1] * 3
        bt.kv_lens = [n + step for n in lens]
        bt.cu, bt.kv_len = np.cumsum([0] + bt.q_lens).astype(np.int32), np.array(bt.kv_lens, np.int32)
        bt.N = int(bt.cu[-1])
        bt.t_cu, bt.t_len = torch.from_numpy(bt.cu).to(DEV), torch.from_numpy(bt.kv_len).to(DEV)
        qkv, x = bf16(g.standard_normal((bt.N, (G + 2) * H, d)))
        pos = np.concatenate([np.arange(n - m, n) for m, n in zip(bt.q_lens, bt.kv_lens)]).astype(np.int32)
        q, k, v = qkv[:, :G * H], qkv[:, G * H:G * H + H], qkv[:, G * H + H:]
        rq.respin_qk_norm_rope(q, k, torch.from_numpy(pos).to(DEV), freq, q, k, q_weight=w, k_weight=w)
        rq.respin_kv_append(bt.cache, k, v, bt.t_len, bt.t_table, cu=bt.t_cu)
        out, _ = attend(_seen(bt, k, v), G * H, q=q.double().cpu().numpy())
        ref, amp = AO.norm_rope(x[:, G * H:G * H + H], w64, 1e-6, pos, freq.cpu().numpy(), False)
        assert (np.abs(k.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * amp).all()


def _seen(bt, k, v):
    """The oracle's cache after the same append; equal to the GPU's."""
    for codes, scale, x, tc, ts in ((bt.kc, bt.ks, k, bt.cache.k, bt.cache.k_scale), (bt.vc, bt.vs, v, bt.cache.v, bt.cache.v_scale)):
        AO.append(codes, scale, x.double().cpu().numpy(), bt.cu, bt.kv_len, bt.table, bt.P)
        assert np.array_equal(tc.cpu().numpy(), codes) and np.array_equal(ts.cpu().numpy(), scale)
    return bt
