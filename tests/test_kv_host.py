"""Host-side checks of the cache and attention calls that need no GPU: bad
arguments are refused before the device is touched."""
import ctypes

import pytest
import torch

import oracle.attention_oracle as AO
import rotation_post_quantization_b200 as rq

# fake, suitably aligned device addresses: validation never dereferences them
A, MIS = 0x10000, 0x10008


def cache(**kw):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, num_pages=4, page_size=16, kv_heads=2, head_dim=64) | kw
    return rq._KvCacheC(**f)


def batch(**kw):
    return rq._KvBatchC(**(dict(cu=None, kv_len=A, block_table=A, B=2, max_pages=3, N=2) | kw))


def attention(c=None, b=None, **kw):
    f = dict(q=A, q_heads=4, ld_q=256, max_q=0, causal=1, window=0, scale=0.125, out=A, ld_out=256, lse=None,
             ws=A, ws_bytes=1 << 40) | kw
    return rq.lib.respin_kv_attention(c or cache(), b or batch(), *f.values(), None)


CACHE = [(dict(head_dim=96), rq.RESPIN_ERR_UNSUPPORTED), (dict(page_size=24), rq.RESPIN_ERR_UNSUPPORTED),
         (dict(kv_heads=0), rq.RESPIN_ERR_UNSUPPORTED), (dict(num_pages=0), rq.RESPIN_ERR_INVALID_ARG),
         (dict(num_pages=1 << 27), rq.RESPIN_ERR_UNSUPPORTED), (dict(k=None), rq.RESPIN_ERR_INVALID_ARG),
         (dict(v_scale=None), rq.RESPIN_ERR_INVALID_ARG), (dict(v=MIS), rq.RESPIN_ERR_ALIGNMENT),
         (dict(k_scale=A + 2), rq.RESPIN_ERR_ALIGNMENT)]
BATCH = [(dict(B=-1), rq.RESPIN_ERR_INVALID_ARG), (dict(N=-1), rq.RESPIN_ERR_INVALID_ARG), (dict(N=3), rq.RESPIN_ERR_INVALID_ARG),
         (dict(B=0), rq.RESPIN_ERR_INVALID_ARG), (dict(max_pages=0), rq.RESPIN_ERR_INVALID_ARG),
         (dict(max_pages=1 << 28), rq.RESPIN_ERR_INVALID_ARG), (dict(B=1 << 20), rq.RESPIN_ERR_UNSUPPORTED),
         (dict(kv_len=None), rq.RESPIN_ERR_INVALID_ARG), (dict(block_table=None), rq.RESPIN_ERR_INVALID_ARG),
         (dict(cu=A + 1), rq.RESPIN_ERR_ALIGNMENT)]


@pytest.mark.parametrize("call", ["append", "read", "attention"])
@pytest.mark.parametrize("kw,want", [(("c", k), w) for k, w in CACHE] + [(("b", k), w) for k, w in BATCH])
def test_cache_and_batch(call, kw, want):
    c, b = (cache(**kw[1]), batch()) if kw[0] == "c" else (cache(), batch(**kw[1]))
    st = (attention(c, b) if call == "attention" else
          getattr(rq.lib, f"respin_kv_{call}")(c, b, A, A, 128, 128, None))
    assert st == want and rq.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), rq.RESPIN_ERR_INVALID_ARG), (dict(out=None), rq.RESPIN_ERR_INVALID_ARG), (dict(ws=None), rq.RESPIN_ERR_INVALID_ARG),
    (dict(q_heads=3), rq.RESPIN_ERR_UNSUPPORTED), (dict(q_heads=0), rq.RESPIN_ERR_UNSUPPORTED), (dict(ld_q=255), rq.RESPIN_ERR_INVALID_ARG),
    (dict(ld_q=128), rq.RESPIN_ERR_INVALID_ARG), (dict(ld_out=260), rq.RESPIN_ERR_INVALID_ARG), (dict(max_q=-1), rq.RESPIN_ERR_INVALID_ARG),
    (dict(window=-1), rq.RESPIN_ERR_INVALID_ARG), (dict(window=5, causal=0), rq.RESPIN_ERR_INVALID_ARG),
    (dict(scale=float("nan")), rq.RESPIN_ERR_INVALID_ARG), (dict(scale=float("inf")), rq.RESPIN_ERR_INVALID_ARG),
    (dict(q=MIS), rq.RESPIN_ERR_ALIGNMENT), (dict(out=MIS), rq.RESPIN_ERR_ALIGNMENT), (dict(lse=A + 1), rq.RESPIN_ERR_ALIGNMENT),
    (dict(ws=MIS), rq.RESPIN_ERR_ALIGNMENT), (dict(ws_bytes=100), rq.RESPIN_ERR_INVALID_ARG)])
def test_attention_arguments(kw, want):
    assert attention(**kw) == want and rq.last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), rq.RESPIN_ERR_INVALID_ARG), (dict(v=MIS), rq.RESPIN_ERR_ALIGNMENT), (dict(ld_k=120), rq.RESPIN_ERR_INVALID_ARG),
    (dict(ld_v=129), rq.RESPIN_ERR_INVALID_ARG)])
def test_append_and_read_arguments(kw, want):
    f = dict(k=A, v=A, ld_k=128, ld_v=128) | kw
    for name in ("respin_kv_append", "respin_kv_read"):
        assert getattr(rq.lib, name)(cache(), batch(), *f.values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), rq.RESPIN_ERR_INVALID_ARG), (dict(d=32), rq.RESPIN_ERR_UNSUPPORTED), (dict(rot=72), rq.RESPIN_ERR_UNSUPPORTED),
    (dict(rot=8), rq.RESPIN_ERR_UNSUPPORTED), (dict(Hq=-1), rq.RESPIN_ERR_UNSUPPORTED), (dict(Hq=0, Hk=0), rq.RESPIN_ERR_UNSUPPORTED),
    (dict(q=None), rq.RESPIN_ERR_INVALID_ARG), (dict(pos=None), rq.RESPIN_ERR_INVALID_ARG), (dict(qw=A, eps=0.0), rq.RESPIN_ERR_INVALID_ARG),
    (dict(qw=A, eps=float("nan")), rq.RESPIN_ERR_INVALID_ARG), (dict(ldq=100), rq.RESPIN_ERR_INVALID_ARG), (dict(qo=MIS), rq.RESPIN_ERR_ALIGNMENT),
    (dict(kw=MIS), rq.RESPIN_ERR_ALIGNMENT), (dict(freq=A + 2), rq.RESPIN_ERR_ALIGNMENT)])
def test_norm_rope_arguments(kw, want):
    f = dict(q=A, k=A, N=2, Hq=4, Hk=2, d=64, ldq=256, ldk=128, qw=None, kw=None, eps=1e-6, pos=A, freq=A, rot=64,
             inter=0, qo=A, ko=A, ldqo=256, ldko=128) | kw
    assert rq.lib.respin_qk_norm_rope(*f.values(), None) == want and rq.last_error()


def test_attention_rows_beyond_32_bits():
    b = batch(N=1 << 30, B=1 << 10)
    assert attention(b=b, q_heads=8, ld_q=512, ld_out=512) == rq.RESPIN_ERR_UNSUPPORTED


def test_empty_calls_do_nothing():
    b = batch(N=0, B=0, kv_len=None, block_table=None)
    assert rq.lib.respin_kv_append(cache(), b, None, None, 0, 0, None) == rq.RESPIN_OK
    assert rq.lib.respin_kv_read(cache(), b, None, None, 0, 0, None) == rq.RESPIN_OK
    assert attention(b=b, q=None, out=None, ws=None) == rq.RESPIN_OK
    assert attention(b=batch(N=0)) == rq.RESPIN_OK


def test_workspace_size():
    n = ctypes.c_longlong(0)
    f = rq.lib.respin_kv_attention_workspace
    assert f(32, 8, 128, 4, 1, ctypes.byref(n)) == rq.RESPIN_OK and n.value > 0
    one = n.value
    assert f(32, 8, 128, 4096, 0, ctypes.byref(n)) == rq.RESPIN_OK and n.value >= one
    assert f(32, 8, 128, 4096, 1, ctypes.byref(n)) == rq.RESPIN_OK and n.value == one
    for bad in ((33, 8, 128, 4, 1), (32, 0, 128, 4, 1), (32, 8, 128, -1, 1), (32, 8, 128, 4, -1)):
        assert f(*bad, ctypes.byref(n)) == rq.RESPIN_ERR_INVALID_ARG
    assert f(32, 8, 80, 4, 1, ctypes.byref(n)) == rq.RESPIN_ERR_UNSUPPORTED
    assert f(32, 8, 128, 4, 1, None) == rq.RESPIN_ERR_INVALID_ARG


def test_launch_fault(monkeypatch):
    monkeypatch.setenv("RESPIN_FAULT", "launch")
    assert attention() == rq.RESPIN_ERR_CUDA and "injected" in rq.last_error()
    assert rq.lib.respin_kv_append(cache(), batch(), A, A, 128, 128, None) == rq.RESPIN_ERR_CUDA
    assert rq.lib.respin_kv_read(cache(), batch(), A, A, 128, 128, None) == rq.RESPIN_ERR_CUDA


def test_binding_refuses_what_the_kernels_would_misread():
    c = rq.KvCache.empty(4, 16, 2, 64, device="cpu")
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    n, t = torch.ones(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="current CUDA device"):
        rq.respin_kv_append(c, x, x, n, t)
    with pytest.raises(ValueError, match="current CUDA device"):
        rq.respin_kv_attention(c, x, n, t, x, torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="current CUDA device"):
        rq.respin_qk_norm_rope(x, x, n, torch.ones(8), x, x)


def test_oracle_quantizer_by_hand():
    """One head, one page: the scale grows with a larger token and moves the earlier codes."""
    import numpy as np
    codes, scale = np.zeros((1, 1, 16, 4), np.int8), np.zeros((1, 1), np.float32)
    table = np.array([[0]])
    AO.append(codes, scale, np.array([[[127.0, -63.5, 1.0, 0.4]]]), [0, 1], [1], table, 16)
    assert scale[0, 0] == 1.0 and codes[0, 0, 0].tolist() == [127, -64, 1, 0]
    AO.append(codes, scale, np.array([[[254.0, 3.0, np.nan, -np.inf]]]), [0, 1], [2], table, 16)
    assert scale[0, 0] == 2.0 and codes[0, 0, 0].tolist() == [64, -32, 0, 0]   # ties to even
    assert codes[0, 0, 1].tolist() == [127, 2, 0, -127]
