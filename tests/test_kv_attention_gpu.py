"""Attention over the 8-bit paged cache against the float64 oracle: head
layouts, lengths from none to many pages, ragged batches, masks that leave a
row empty, and the call's use (streams, graphs, strides, refused indexes)."""
import numpy as np
import pytest
import torch

import rotation_post_quantization_b200 as rq
from kv_util import DEV, Batch, attend, bf16, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (2, 4), (1, 8), (2, 7)])
def test_decode(H, G, d, P):
    lens = [1, 15, 16, 17, 63, 64, 65, 200, 0, 333]
    bt = Batch([1] * len(lens), lens, H, d, P, seed=H * 100 + G).to_gpu()
    attend(bt, H * G, use_cu=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 4])
def test_ragged_rows(G, d):
    """Chunks of 0 to 40 rows, some of them longer than their sequence's start, rows behind the last sequence."""
    q, kv = [3, 0, 1, 40, 5, 17, 2], [3, 50, 129, 40, 300, 260, 2]
    bt = Batch(q, kv, 2, d, 32, seed=G, behind=5).to_gpu()
    attend(bt, 2 * G)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 1000])
def test_window(window):
    bt = Batch([1, 30, 7, 1], [500, 200, 9, 64], 2, 128, 16, seed=window).to_gpu()
    attend(bt, 8, window=window)


def test_not_causal():
    bt = Batch([1, 30, 7, 2], [500, 200, 9, 0], 2, 64, 64, seed=4).to_gpu()
    attend(bt, 4, causal=False)


@pytest.mark.parametrize("q", [1, 9, 70])
def test_empty_rows(q):
    """More rows than the sequence has tokens: the first ones see nothing."""
    bt = Batch([q, q, q], [0, q // 2 + 1, q], 1, 128, 16, seed=q).to_gpu()
    out, lse = attend(bt, 4)
    assert (lse[:q] == -np.inf).all()


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [20000, 131]), ([1], [70001]), ([2, 1, 8], [30000, 1, 9000])])
def test_long_contexts_are_split(q_lens, kv_lens):
    bt = Batch(q_lens, kv_lens, 2, 128, 128, seed=8).to_gpu()
    attend(bt, 16)


@pytest.mark.parametrize("H,G,d,q,kv", [(2, 4, 128, 300, 300), (1, 1, 64, 513, 900), (2, 8, 64, 129, 2000),
                                        (4, 1, 128, 256, 256), (1, 3, 128, 333, 5000)])
def test_prefill(H, G, d, q, kv):
    bt = Batch([q], [kv], H, d, 64, seed=q).to_gpu()
    attend(bt, H * G)


@pytest.mark.parametrize("window,causal", [(0, True), (37, True), (700, True), (0, False)])
def test_prefill_ragged_masks(window, causal):
    bt = Batch([200, 1, 0, 65, 400], [900, 2000, 10, 65, 1200], 2, 128, 16, seed=window, behind=3).to_gpu()
    attend(bt, 8, window=window, causal=causal)


@pytest.mark.parametrize("q", [1, 60])
def test_value_scales_of_pages_far_apart(q):
    """Pages whose value scales differ by up to 2^24, one page of zeros: the
    weights carry the scale, so a small page beside a large one must not lose
    the row's sum."""
    bt = Batch([q], [640], 2, 128, 64, seed=5, v_spread=12.0)
    z = bt.table[0, 3]
    bt.vc[z] = 0
    bt.vs[z] = 0.0
    attend(bt.to_gpu(), 4)


@pytest.mark.parametrize("q", [1, 60])
@pytest.mark.parametrize("gain", [1e-30, 30.0, 2.0 ** 60])
def test_query_sizes(gain, q):
    """Logits near zero, peaked ones, and queries whose size only the scale brings back."""
    bt = Batch([q], [300], 1, 128, 32, seed=6).to_gpu()
    attend(bt, 4, q_gain=gain, scale=None if gain < 1e3 else 2.0 ** -62)


def test_zero_queries_and_keys():
    bt = Batch([1, 50], [100, 80], 1, 64, 16, seed=7)
    bt.kc[:] = 0
    attend(bt.to_gpu(), 2, q=np.zeros((51, 2, 64)))


def test_unwritten_slots_do_not_matter():
    """Bytes behind the last token, in and behind the last page, and pages of nobody."""
    bt = Batch([1, 33], [70, 40], 2, 128, 64, seed=9).to_gpu()
    a = attend(bt, 8)
    used = {(int(p), s) for b in range(2) for t in range(bt.kv_lens[b]) for p, s in [(bt.table[b, t // 64], t % 64)]}
    m = np.array([[(p, s) not in used for s in range(64)] for p in range(bt.pages)])
    for c in (bt.cache.k, bt.cache.v):
        c[torch.from_numpy(m)[:, None, :, None].expand(c.shape).to(DEV)] = 101
    for p in range(bt.pages):
        if not any((p, s) in used for s in range(64)):
            bt.cache.k_scale[p] = float("nan")
            bt.cache.v_scale[p] = float("inf")
    b = attend(bt, 8)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_strided_query_and_output():
    bt = Batch([1, 40], [100, 77], 2, 128, 32, seed=10).to_gpu()
    wide = torch.randn(41, 16, 128, device=DEV).bfloat16()
    q = wide[:, 3:11]
    to = torch.zeros(41, 12, 128, dtype=torch.bfloat16, device=DEV)
    ws = workspace(bt.cache, 8, 41)
    rq.respin_kv_attention(bt.cache, q, bt.t_len, bt.t_table, to[:, 2:10], ws, cu=bt.t_cu)
    want, _ = attend(bt, 8, q=q.double().cpu().numpy(), max_q=None)
    assert torch.equal(to[:, 2:10], want) and (to[:, :2] == 0).all() and (to[:, 10:] == 0).all()


def test_repeated_and_on_streams():
    """The same bits again, eagerly, on two streams at once, and from a graph
    replayed after the lengths changed in place."""
    bt = Batch([1, 1, 1], [3000, 77, 900], 2, 128, 64, seed=11).to_gpu()
    tq, _ = bf16(np.random.default_rng(3).standard_normal((3, 8, 128)))
    outs = [torch.zeros(3, 8, 128, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    wss = [workspace(bt.cache, 8, 3, 1) for _ in range(3)]

    def call(i):
        rq.respin_kv_attention(bt.cache, tq, bt.t_len, bt.t_table, outs[i], wss[i])

    call(0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                call(i + 1)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(1)
    bt.t_len.copy_(torch.tensor([64, 77, 2999], dtype=torch.int32))
    bt.t_table[2] = bt.t_table[0].clone()   # any pages will do
    call(0)
    g.replay()
    torch.cuda.synchronize()
    assert rq.respin_device_status() == 0
    assert torch.equal(outs[0], outs[1]) and not torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("q", [1, 50])
def test_refused_indexes_are_recorded(q):
    """A page id outside the cache leaves its tokens out; a length beyond the
    table, or a cu that does not fit, leaves the sequence out: the other's rows are those of a
    batch without it (to the bit: the same line of work; beside a sequence that counts, the
    order of a shared unit's sums may be another)."""
    bt = Batch([q, q], [200, 200], 1, 128, 64, seed=12).to_gpu()
    tq, _ = bf16(np.random.default_rng(3).standard_normal((2 * q, 4, 128)))
    ws = workspace(bt.cache, 4, 2 * q)

    def call():
        out = torch.full((2 * q, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        rq.respin_kv_attention(bt.cache, tq, bt.t_len, bt.t_table, out, ws, cu=bt.t_cu, max_q=q)
        return out

    good = call()
    assert rq.respin_device_status() == 0
    for bad in (-5, bt.pages, 2 ** 31 - 1):
        keep = bt.t_table.clone()
        bt.t_table[0, 1] = bad
        got = call()
        assert rq.respin_device_status() == 511
        assert torch.equal(got[q:], good[q:]) and not torch.isnan(got).any()
        bt.t_table.copy_(keep)
    bt.t_cu[0] = q   # no rows of the first sequence
    alone = call()
    assert rq.respin_device_status() == 0 and (alone[:q] == 7).all()
    bt.t_cu[0] = 0
    for t, i, bad in ((bt.t_len, 0, 10 ** 6), (bt.t_len, 0, -1), (bt.t_cu, 0, -3), (bt.t_cu, 0, 2 * q + 9)):
        keep = t.clone()
        t[i] = bad
        got = call()
        assert rq.respin_device_status() == 512
        assert torch.equal(got[q:], alone[q:]) and (got[:q] == 7).all()
        t.copy_(keep)
    assert torch.equal(call(), good)
    assert rq.respin_device_status() == 0

def test_max_q_below_the_truth_is_recorded():
    bt = Batch([1, 40], [100, 77], 1, 128, 32, seed=13).to_gpu()
    tq, _ = bf16(np.random.default_rng(3).standard_normal((41, 4, 128)))
    out = torch.full((41, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    rq.respin_kv_attention(bt.cache, tq, bt.t_len, bt.t_table, out, workspace(bt.cache, 4, 41, 2), cu=bt.t_cu, max_q=2)
    assert rq.respin_device_status() == 512
    assert (out[1:] == 7).all() and not (out[:1] == 7).all()


@pytest.mark.parametrize("q", [1, 3, 40])
@pytest.mark.parametrize("P", [16, 64, 128])
def test_pages_behind_the_window_may_be_gone(q, P):
    """A sliding window's freed pages have no id any more: not looked at, nothing recorded."""
    bt = Batch([q, q], [700, 300], 2, 128, P, seed=14).to_gpu()
    want = attend(bt, 8, window=100)
    for b, n in enumerate(bt.kv_lens):
        gone = max(0, n - q - 100 + 1) // P   # pages that no row's window touches
        assert gone > 0
        bt.t_table[b, :gone] = -1
    got = attend(bt, 8, window=100)
    assert all(torch.equal(x, y) for x, y in zip(want, got))


@pytest.mark.parametrize("q", [1, 50])
@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_scale_negative_or_zero(scale, q):
    bt = Batch([q], [300], 2, 128, 32, seed=15).to_gpu()
    attend(bt, 4, scale=scale)


@pytest.mark.parametrize("H,G,q", [(1, 16, 1), (1, 17, 1), (1, 64, 3), (2, 32, 9), (1, 5, 300)])
def test_many_query_heads_of_a_key_head(H, G, q):
    bt = Batch([q, q], [400, q + 1], H, 64, 64, seed=16).to_gpu()
    attend(bt, H * G)


@pytest.mark.parametrize("q", [2, 60])
def test_a_row_of_nan_stays_alone(q):
    bt = Batch([q], [200], 1, 128, 64, seed=17).to_gpu()
    x = np.random.default_rng(4).standard_normal((q, 4, 128))
    tq, _ = bf16(x)
    ws = workspace(bt.cache, 4, q)
    outs = []
    for bad in (None, float("nan"), float("inf")):
        t = tq.clone()
        if bad is not None:
            t[1, 2, 5] = bad
        out = torch.zeros_like(tq)
        rq.respin_kv_attention(bt.cache, t, bt.t_len, bt.t_table, out, ws)
        outs.append(out)
    for o in outs[1:]:
        assert torch.isnan(o[1, 2]).all()
        o[1, 2] = outs[0][1, 2]
        assert torch.equal(o, outs[0])


def test_window_beyond_any_length():
    bt = Batch([40, 1], [30, 500], 1, 64, 16, seed=18).to_gpu()
    a = attend(bt, 2)
    for window in (2 ** 31 - 1, 16 * bt.table.shape[1]):
        q = np.random.default_rng(1).standard_normal((bt.N, 2, 64))
        out, lse = torch.zeros_like(a[0]), torch.zeros_like(a[1])
        rq.respin_kv_attention(bt.cache, bf16(q)[0], bt.t_len, bt.t_table, out, workspace(bt.cache, 2, bt.N), cu=bt.t_cu,
                               window=window, lse=lse)
        assert torch.equal(out, a[0]) and torch.equal(lse, a[1])


@pytest.mark.parametrize("q", [1, 40])
def test_c_call_without_cu_and_max_q(q):
    """N / B rows each and no max_q: as if it had been given."""
    bt = Batch([q, q], [100, 77], 1, 128, 32, seed=19).to_gpu()
    want, _ = attend(bt, 4)
    tq, _ = bf16(np.random.default_rng(1).standard_normal((2 * q, 4, 128)))
    c, b, _ = rq._kv_args(bt.cache, 2 * q, bt.t_len, bt.t_table, None)
    out, ws = torch.zeros_like(tq), workspace(bt.cache, 4, 2 * q)
    rq._check(rq.lib.respin_kv_attention(c, b, tq.data_ptr(), 4, 512, 0, 1, 0, 128 ** -0.5, out.data_ptr(), 512, None,
                                         ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert rq.respin_device_status() == 0 and torch.equal(out, want)


def test_padded_batch():
    """Sequences without rows, as a graph of a fixed batch size pads with: whatever their length and pages say."""
    bt = Batch([1, 40, 0, 0], [100, 77, 5, 5], 1, 128, 32, seed=20).to_gpu()
    a = attend(bt, 4)
    bt.t_len[2:] = torch.tensor([-7, 10 ** 9], dtype=torch.int32)
    bt.t_table[2:] = -1
    b = attend(bt, 4)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    k = torch.zeros(41, 1, 128, dtype=torch.bfloat16, device=DEV)
    rq.respin_kv_append(bt.cache, k, k, bt.t_len, bt.t_table, cu=bt.t_cu)
    rq.respin_kv_read(bt.cache, k, k.clone(), bt.t_len, bt.t_table, cu=bt.t_cu)
    assert rq.respin_device_status() == 0
